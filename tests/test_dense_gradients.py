"""The dense block's gradients along directions, against central differences of the 64-bit forward
pass: directions aligned with the gradient (all of it, and stretches of its rows), so that a term
that is missing or counted twice changes <gradient, direction> by a share of its value, and a
tolerance from independent roundings, which is a few thousandths of that value.

Tolerance. The kernels round h, dg, du and the results to 16 bits, each value by at most half a
step, independently: uniform errors of at most half |v_i| give a weighted sum with a standard
deviation of half / sqrt(3) times the 2-norm of the weighted values, and the bound is four such
norms (6.9 standard deviations). The weights of an intermediate's error in <gradient, direction> are
the direction times the operand it is multiplied with. What is rounded to fp32 (sums, activations)
may err in one direction, so its worst-case bound counts in full: that of ffn_ref with
intermediates and results of fp32.
"""
import pytest

torch = pytest.importorskip("torch")
from dense_helpers import HALF_STEP, activation, ffn_ref

BF, HF = torch.bfloat16, torch.float16
NAMES = ("dx", "dw_gate", "dw_up", "dw_down")
SHAPES = [(96, 136, 200), (33, 264, 72), (300, 520, 264)]


def problem(T, d, f, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    shapes = ((T, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5), (d, f, f ** -0.5), (T, d, 0.5))
    return [(torch.randn(r, c, generator=gen) * s).to(dtype) for r, c, s in shapes]


def backward(x, wg, wu, wd, dy, act, rounded=lambda t: t, drop=None):
    """The four gradients in 64 bits, intermediates and results passed through `rounded`; `drop`
    names a term to leave out (a mistake planted in the oracle)."""
    g, u, dh = x @ wg.T, x @ wu.T, dy @ wd
    a, da = activation(g, act)
    if drop == "slope":                             # act'(g) taken as act(g) / g
        da = a / g
    h, dg, du = rounded(a * u), rounded(dh * u * da), rounded(dh * a)
    parts = [dg @ wg, du @ wu]
    if drop in (0, 1):
        parts[drop] = 0 * parts[drop]
    last = slice(0, x.shape[0] - 32 if drop == "rows" else None)
    return [rounded(t) for t in (parts[0] + parts[1], dg[last].T @ x[last], du[last].T @ x[last],
                                 dy[last].T @ h[last])]


def directions(ref):
    """Unit vectors along the gradient, whole and in quarters of its rows."""
    n = ref.shape[0]
    yield ref / ref.norm()
    for q in range(4):
        v = torch.zeros_like(ref)
        v[q * n // 4:(q + 1) * n // 4] = ref[q * n // 4:(q + 1) * n // 4]
        yield v / v.norm()


def worst(grads, x, wg, wu, wd, dy, act, dtype):
    """{name: (largest |<gradient, v> - difference| / tolerance, largest tolerance / |difference|)}."""
    half = HALF_STEP[dtype]
    inputs = [t.double() for t in (x, wg, wu, wd)]
    x, wg, wu, wd = inputs
    dy = dy.double()
    ref = ffn_ref(x, wg, wu, wd, act, torch.float32, dy=dy)
    g, u, dh = x @ wg.T, x @ wu.T, dy @ wd
    a, da = activation(g, act)
    h, dg, du = a * u, dh * u * da, dh * a

    def loss(v):
        return ((activation(v[0] @ v[1].T, act)[0] * (v[0] @ v[2].T)) @ v[3].T * dy).sum()

    out = {}
    for i, (name, grad) in enumerate(zip(NAMES, grads)):
        value, bound = ref[name]
        ratios, shares = [], []
        for v in directions(value):
            weighted = {"dx": lambda: (dg * (v @ wg.T), du * (v @ wu.T)),
                        "dw_gate": lambda: (dg * (x @ v.T),),
                        "dw_up": lambda: (du * (x @ v.T),),
                        "dw_down": lambda: (h * (dy @ v),)}[name]()
            rounding = sum(t.square().sum() for t in (value * v, *weighted)).sqrt()
            tol = (4 * half * rounding + (bound * v.abs()).sum()).item()
            e = 1e-4
            plus, minus = (loss([t + s * e * v if j == i else t for j, t in enumerate(inputs)])
                           for s in (1, -1))
            diff = ((plus - minus) / (2 * e)).item()
            # (truncation of order e^2 with |v| = 1, rounding 2^-52 |loss| / e)
            got = (grad.double().to(v.device) * v).sum().item()
            ratios.append(abs(got - diff) / (tol + 1e-6 * abs(diff)))
            shares.append(tol / abs(diff))
        out[name] = max(ratios), max(shares)
    return out


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_check_accepts_roundings_and_rejects_mistakes(act, dtype):
    """The check itself, on gradients made here: rounded where the kernels round it accepts them;
    zeroed, halved, with a term or the last 32 rows left out, or with a wrong slope it does not."""
    for T, d, f in SHAPES:
        p = problem(T, d, f, dtype, T)
        v64 = [t.double() for t in p]
        make = lambda drop=None: backward(*v64, act, lambda t: t.to(dtype).double(), drop)  # noqa: E731
        good = make()
        for name, (ratio, share) in worst(good, *p, act, dtype).items():
            assert ratio <= 1 and share < 0.02, (name, ratio, share)
        for bad, which in (([0 * t for t in good], NAMES), ([t / 2 for t in good], NAMES),
                           ([t * 1.1 for t in good], NAMES), (make(0), ("dx",)), (make(1), ("dx",)),
                           (make("rows"), NAMES[1:]), (make("slope"), ("dw_gate",))):
            got = worst(bad, *p, act, dtype)
            for name in which:
                assert got[name][0] > 1, (name, got[name])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_gradients_along_themselves_match_differences(T, d, f, dtype, act):
    from expert_routed_ffn_route_b200 import binding as B
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, wg, wu, wd, dy = (t.cuda() for t in problem(T, d, f, dtype, T))
    bank = dict(fmt="bf16" if dtype == BF else "fp16", w_gate=wg, w_up=wu, w_down=wd)
    block = B.DeviceFfn(bank, d, f, act=act)
    desc = block.descriptor(T)
    ws, pre = B.alloc_ffn_workspace(desc, backward=True), B.ffn_pre(desc)
    B.ffn_forward(desc, x, ws, pre=pre)
    grads = B.ffn_backward(desc, x, dy, pre, ws)
    for name, (ratio, _) in worst(grads, x, wg, wu, wd, dy, act, dtype).items():
        assert ratio <= 1, (name, ratio)
