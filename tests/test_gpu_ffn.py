"""The dense gated block on the GPU, forward and backward, against a plain implementation in 64
bits and against differences."""
import pytest

torch = pytest.importorskip("torch")
from dense_helpers import (TINY, activation, assert_close, assert_norm_close, dequantise, ffn_ref,
                           matvec_additions, matvec_ref, quantise)

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
FMT = {BF: "bf16", HF: "fp16"}


@pytest.fixture(scope="module")
def B():
    from expert_routed_ffn_route_b200 import binding
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()
    return binding


def make(B, d, f, dtype=BF, act="silu", seed=0, fmt=None):
    """A block on the GPU and its weights in 64 bits."""
    gen = torch.Generator().manual_seed(seed)
    bank, W = dict(fmt=fmt or FMT[dtype], group=128, n_exp=1), []
    for m, N, K in (("gate", f, d), ("up", f, d), ("down", d, f)):
        if fmt == "int4":
            codes, scales = quantise(gen, N, K, 128)
            bank["w_" + m], bank["s_" + m] = codes.cuda(), scales.cuda()
            W.append(dequantise(codes, scales, 128).cuda())
        else:
            w = (torch.randn(N, K, generator=gen) * K ** -0.5).to(dtype).cuda()
            bank["w_" + m] = w
            W.append(w.double())
    return B.DeviceFfn(bank, d, f, act=act), W


def rows(T, d, dtype, seed=1, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, d, generator=gen) * scale).to(dtype).cuda()


def guarded(T, cols, dtype):
    """[T, cols] inside a larger buffer whose rest must stay as it was."""
    buf = torch.full((T * cols + 256,), 3.0, dtype=dtype, device="cuda")
    return buf, buf[:T * cols].view(T, cols)


# T, d, f: single rows and values, tails in every direction of the 128 x (64, 128, 256) x 64 tiles
SHAPES = [
    (1, 8, 8), (1, 128, 256), (2, 264, 72), (7, 136, 520), (31, 1024, 264), (32, 512, 1032),
    (33, 8, 16), (33, 136, 72), (64, 2560, 1024), (100, 72, 2056), (127, 64, 64),
    (128, 128, 128), (129, 256, 264), (257, 1032, 136), (300, 520, 1032), (700, 1288, 1160),
    (2049, 640, 392),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_forward_matches_64_bits(B, T, d, f, act, dtype):
    block, W = make(B, d, f, dtype, act, seed=d + f)
    x = rows(T, d, dtype)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc)
    buf, y = guarded(T, d, dtype)
    B.ffn_forward(desc, x, ws, out=y)
    pbuf, pre = guarded(2 * T, f, F32)
    pre = pre.view(2, T, f)
    tws = B.alloc_ffn_workspace(desc, backward=True)
    y2 = B.ffn_forward(desc, x, tws, pre=pre)
    assert B.ffn_device_status(desc, ws) == (0, 0) and B.ffn_device_status(desc, tws) == (0, 0)
    ref, bound = ffn_ref(x, *W, act, dtype)["y"]
    for out in (y, y2):
        assert_close(out, ref, bound, dtype, "y")
        assert_norm_close(out, ref, dtype, "y")
    assert (buf[T * d:] == 3).all() and (pbuf[2 * T * f:] == 3).all()
    xd = x.double()
    for got, w in zip(pre, W[:2]):
        r, mag = matvec_ref(xd, w)
        assert_close(got, r, mag * (d // 8 + 64) * 2.0 ** -23, F32, "pre")
    if T > 32:  # the same kernels with and without pre
        assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype,act", [(BF, "silu"), (HF, "gelu"), (BF, "gelu"), (HF, "silu")])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_backward_matches_64_bits(B, T, d, f, act, dtype):
    block, W = make(B, d, f, dtype, act, seed=d + f + 1)
    x, dy = rows(T, d, dtype), rows(T, d, dtype, seed=2, scale=0.5)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc, backward=True)
    pre = B.ffn_pre(desc)
    B.ffn_forward(desc, x, ws, pre=pre)
    names = ("dx", "dw_gate", "dw_up", "dw_down")
    got = dict(zip(names, B.ffn_backward(desc, x, dy, pre, ws)))
    again = dict(zip(names, B.ffn_backward(desc, x, dy, pre, ws)))
    assert B.ffn_device_status(desc, ws) == (0, 0)
    ref = ffn_ref(x, *W, act, dtype, dy=dy)
    for n in names:
        assert torch.equal(got[n], again[n]), n
        assert_close(got[n], *ref[n], dtype, n)
        assert_norm_close(got[n], ref[n][0], dtype, n)


def test_calls_of_any_kind_share_one_workspace_in_turn(B):
    """Streamed and tensor-core calls, forward and backward, of blocks and matrices of several
    sizes use one workspace one after the other; every result has the bits that a workspace of its
    own gives (what one call leaves behind is nothing that another counts on)."""
    gen = torch.Generator().manual_seed(5)
    calls = []
    for T, d, f in ((1, 2560, 1024), (16, 1024, 2056), (32, 2560, 1024), (40, 512, 1032), (4, 72, 4096)):
        block, _ = make(B, d, f, seed=T)
        desc, x, dy = block.descriptor(T), rows(T, d, BF, T), rows(T, d, BF, T + 1)

        def train(ws, desc=desc, x=x, dy=dy):
            pre = B.ffn_pre(desc)
            y = B.ffn_forward(desc, x, ws, pre=pre)
            return (y, *B.ffn_backward(desc, x, dy, pre, ws))
        calls.append((lambda ws, desc=desc, x=x: (B.ffn_forward(desc, x, ws),),
                      B.alloc_ffn_workspace(desc)))
        calls.append((train, B.alloc_ffn_workspace(desc, backward=True)))
    for T, N, K in ((32, 1000, 10240), (16, 2560, 10240), (1, 77, 256)):
        codes, scales = quantise(gen, N, K, 32)
        desc = B.QuantMatrix(codes.cuda(), scales.cuda(), K, 32).descriptor(T)
        calls.append((lambda ws, desc=desc, x=rows(T, K, BF, N): (B.matvec(desc, x, ws),),
                      B.alloc_matvec_workspace(desc)))
    own = [fn(ws) for fn, ws in calls]
    shared = torch.zeros(max(ws.numel() for _, ws in calls), dtype=torch.uint8, device="cuda")
    n = len(calls)
    for i in range(n):
        for j in range(n):                         # each call after each other one
            for k in (i, j):
                got = calls[k][0](shared)
                assert all(torch.equal(a, b) for a, b in zip(got, own[k])), (i, j, k)


def test_a_long_step_repeats_bit_for_bit(B):
    """A step large enough to keep every SM busy (copies then arrive while others are still being
    read), many times over: every result the same bits, and those of the reference."""
    T, d, f = 2048, 1024, 8192
    block, W = make(B, d, f)
    x, dy = rows(T, d, BF), rows(T, d, BF, seed=2, scale=0.5)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc, backward=True)
    names = ("y", "pre", "dx", "dw_gate", "dw_up", "dw_down")

    def step():
        pre = B.ffn_pre(desc)
        y = B.ffn_forward(desc, x, ws, pre=pre)
        return dict(zip(names, (y, pre, *B.ffn_backward(desc, x, dy, pre, ws))))
    first = step()
    for _ in range(40):
        again = [step() for _ in range(3)][-1]
        for n in names:
            assert torch.equal(again[n], first[n]), n
    ref = ffn_ref(x, *W, "silu", BF, dy=dy)
    for n in ("y", "dx", "dw_gate", "dw_up", "dw_down"):
        assert_close(first[n], *ref[n], BF, n)
        assert_norm_close(first[n], ref[n][0], BF, n)


def test_the_most_rows(B):
    """2^20 rows: h, dg and du have more than 2^31 values, the kept g and u more than 2^34 bytes. dy
    is zero but in three stretches (the first rows, some in the middle, the last), so that the
    weights' gradients are sums over those alone: the other rows add exact zeros."""
    T, d, f = 1 << 20, 16, 2056
    block, W = make(B, d, f)
    desc = block.descriptor(T)
    at = torch.cat([torch.arange(s, s + 150) for s in (0, T // 2 - 70, T - 150)]).cuda()
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, d, generator=gen, device="cuda").to(BF)
    dy = torch.zeros(T, d, dtype=BF, device="cuda")
    dy[at] = rows(len(at), d, BF, seed=4)
    ws, pre = B.alloc_ffn_workspace(desc, backward=True), B.ffn_pre(desc)
    y = B.ffn_forward(desc, x, ws, pre=pre)
    dx, *dw = B.ffn_backward(desc, x, dy, pre, ws)
    assert B.ffn_device_status(desc, ws) == (0, 0)
    del pre, ws
    ref = ffn_ref(x[at], *W, "silu", BF, dy=dy[at])
    for n, got in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y[at], dx[at], *dw)):
        assert_close(got, *ref[n], BF, n)
        assert_norm_close(got, ref[n][0], BF, n)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (dx[rest] == 0).all()


def test_only_what_is_asked_for_is_computed(B):
    T, d, f = 200, 136, 264
    block, W = make(B, d, f)
    x, dy = rows(T, d, BF), rows(T, d, BF, seed=2)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc, backward=True)
    pre = B.ffn_pre(desc)
    B.ffn_forward(desc, x, ws, pre=pre)
    full = B.ffn_backward(desc, x, dy, pre, ws)
    dx, *none = B.ffn_backward(desc, x, dy, pre, ws, need_dw=False)
    assert none == [None] * 3 and torch.equal(dx, full[0])
    none, *dws = B.ffn_backward(desc, x, dy, pre, ws, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dws, full[1:]))
    with pytest.raises(B.MoeError):
        B.ffn_backward(desc, x, dy, pre, ws, need_dx=False, need_dw=False)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_match_differences(B, act):
    """<gradient, direction> against central differences of the 64-bit forward pass: step e
    gives a truncation error of order e^2 and a rounding error of order 2^-52 / e, both below
    1e-9; what remains is the kernels' 16-bit rounding, bounded by the gradient's own."""
    T, d, f = 96, 136, 200
    block, W = make(B, d, f, HF, act)
    x, dy = rows(T, d, HF), rows(T, d, HF, seed=2)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc, backward=True)
    pre = B.ffn_pre(desc)
    B.ffn_forward(desc, x, ws, pre=pre)
    grads = B.ffn_backward(desc, x, dy, pre, ws)
    inputs = [x.double()] + W

    def loss(v):
        g, u = v[0] @ v[1].T, v[0] @ v[2].T
        return ((activation(g, act)[0] * u) @ v[3].T * dy.double()).sum()

    ref = ffn_ref(x, *W, act, HF, dy=dy)
    gen = torch.Generator(device="cuda").manual_seed(7)
    for i, (name, grad) in enumerate(zip(("dx", "dw_gate", "dw_up", "dw_down"), grads)):
        v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-5
        plus, minus = (loss([t + s * e * v if j == i else t for j, t in enumerate(inputs)])
                       for s in (1, -1))
        diff = ((plus - minus) / (2 * e)).item()
        tol = ((ref[name][1] + grad.double().abs() * 2.0 ** -11 + TINY[HF]) * v.abs()).sum().item()
        assert abs((grad.double() * v).sum().item() - diff) <= tol + 1e-6 * abs(diff), name


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,d,f", [(1, 128, 128), (1, 2560, 1024), (3, 256, 384), (8, 640, 256),
                                   (9, 384, 1280), (16, 2560, 512), (17, 128, 2560), (2, 2560, 4096), (7, 4096, 2560),
                                   (32, 2560, 2560)])
def test_int4_block_matches_64_bits(B, T, d, f, act):
    block, W = make(B, d, f, fmt="int4", act=act, seed=d + f)
    x = rows(T, d, BF)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc)
    buf, y = guarded(T, d, BF)
    B.ffn_forward(desc, x, ws, out=y)
    assert torch.equal(y, B.ffn_forward(desc, x, ws))
    ref, bound = ffn_ref(x, *W, act, BF)["y"]
    assert_close(y, ref, bound, BF, "y")
    assert_norm_close(y, ref, BF, "y")
    assert (buf[T * d:] == 3).all()


@pytest.mark.parametrize("T,d,f,fmt", [(32, 32768, 136, None), (3, 136, 32768, None),
                                       (32, 32768, 128, "int4"), (40, 32768, 72, None)])
def test_the_longest_rows(B, T, d, f, fmt):
    """The widest blocks: rows that are split into K parts, in both products."""
    block, W = make(B, d, f, fmt=fmt, seed=d)
    x = rows(T, d, BF)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc)
    y = B.ffn_forward(desc, x, ws)
    assert torch.equal(y, B.ffn_forward(desc, x, ws))
    ref, bound = ffn_ref(x, *W, "silu", BF)["y"]
    assert_close(y, ref, bound, BF, "y")
    assert_norm_close(y, ref, BF, "y")
    assert B.ffn_device_status(desc, ws) == (0, 0)


@pytest.mark.parametrize("fmt,dtype", [("int4", BF), (None, BF), (None, HF)])
@pytest.mark.parametrize("T,d,f", [(1, 256, 256), (1, 2560, 1024), (3, 384, 2560), (4, 4096, 2560)])
def test_few_rows_round_once(B, T, d, f, fmt, dtype):
    """Up to four streamed rows carry h as its rounded value and the rounded rest (a half step of
    a half step), so y is off by its own rounding and that."""
    block, W = make(B, d, f, dtype, fmt=fmt, seed=T + d)
    x = rows(T, d, dtype)
    desc = block.descriptor(T)
    ws = B.alloc_ffn_workspace(desc)
    half = torch.finfo(dtype).eps / 2
    buf, y = guarded(T, d, dtype)
    B.ffn_forward(desc, x, ws, out=y)
    ref, bound = ffn_ref(x, *W, "silu", dtype, h_half=half * half)["y"]
    assert_close(y, ref, bound, dtype, "y")
    assert (buf[T * d:] == 3).all()
    # one rounding of y, and fp32 sums: the 2-norm of the error is below one half step
    assert ((y.double() - ref).norm() / ref.norm()).item() <= half


def test_a_gate_beyond_fp16_gives_infinity_not_nan(B):
    """h beyond fp16's largest value is infinite, with no rest, and so is y where Wd is not zero."""
    d = f = 128
    bank = dict(fmt="fp16", group=128, n_exp=1,
                w_gate=torch.full((f, d), 30.0, dtype=HF, device="cuda"),
                w_up=torch.full((f, d), 30.0, dtype=HF, device="cuda"),
                w_down=torch.eye(d, dtype=HF, device="cuda") + 1)
    block = B.DeviceFfn(bank, d, f)
    for T in (1, 40):
        desc = block.descriptor(T)
        y = B.ffn_forward(desc, torch.ones(T, d, dtype=HF, device="cuda"), B.alloc_ffn_workspace(desc))
        assert (y == float("inf")).all()


def test_gates_far_from_zero(B):
    """Saturated gates: silu and gelu give g or 0 (never NaN), their slopes 1 or 0."""
    T, d, f = 64, 64, 64
    for act in ("silu", "gelu"):
        block, W = make(B, d, f, BF, act)
        x = rows(T, d, BF, scale=3e4)
        dy = rows(T, d, BF, seed=2)
        desc = block.descriptor(T)
        ws = B.alloc_ffn_workspace(desc, backward=True)
        pre = B.ffn_pre(desc)
        y = B.ffn_forward(desc, x, ws, pre=pre)
        grads = B.ffn_backward(desc, x, dy, pre, ws)
        g, u = pre[0].double(), pre[1].double()
        sat = g.abs() > 100
        assert sat.float().mean() > 0.9
        for t in (y, *grads):
            assert torch.isfinite(t).all()
        a, da = g.clamp_min(0), (g > 0).double()
        h = torch.where(sat, a * u, activation(g, act)[0] * u)
        assert_norm_close(y, h @ W[2].T, BF, act)
        dh = dy.double() @ W[2]
        slope = torch.where(sat, da, activation(g, act)[1])
        act_v = torch.where(sat, a, activation(g, act)[0])
        assert_norm_close(grads[1], (dh * u * slope).T @ x.double(), BF, act)
        assert_norm_close(grads[2], (dh * act_v).T @ x.double(), BF, act)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_a_nan_row_stays_alone(B, T):
    block, W = make(B, 256, 384)
    x = rows(T, 256, BF)
    x[T // 2, 5] = float("nan")
    desc = block.descriptor(T)
    y = B.ffn_forward(desc, x, B.alloc_ffn_workspace(desc))
    assert torch.isnan(y[T // 2]).all()
    keep = [t for t in range(T) if t != T // 2]
    if keep:
        ref, bound = ffn_ref(x[keep], *W, "silu", BF)["y"]
        assert_close(y[keep], ref, bound, BF)


def test_captured_step_replayed_beside_another(B):
    """A training step captured into a graph, two of them with their own workspaces replayed at
    once on two streams."""
    T, d, f = 150, 264, 392
    steps = []
    for seed in (1, 2):
        block, W = make(B, d, f, seed=seed)
        x, dy = rows(T, d, BF, seed), rows(T, d, BF, seed + 10)
        desc = block.descriptor(T)
        c = dict(desc=desc, block=block, W=W, x=x, dy=dy, s=torch.cuda.Stream(), g=torch.cuda.CUDAGraph(),
                 ws=B.alloc_ffn_workspace(desc, backward=True), pre=B.ffn_pre(desc))

        def step(c=c):
            c["y"] = B.ffn_forward(c["desc"], c["x"], c["ws"], pre=c["pre"])
            c["grads"] = B.ffn_backward(c["desc"], c["x"], c["dy"], c["pre"], c["ws"])
        step()
        torch.cuda.synchronize()
        c["eager"] = [t.clone() for t in (c["y"], *c["grads"])]
        with torch.cuda.graph(c["g"], stream=c["s"]):
            step()
        steps.append(c)
    for _ in range(10):
        for c in steps:
            with torch.cuda.stream(c["s"]):
                c["g"].replay()
    torch.cuda.synchronize()
    for c in steps:
        for a, b in zip((c["y"], *c["grads"]), c["eager"]):
            assert torch.equal(a, b)
        assert B.ffn_device_status(c["desc"], c["ws"]) == (0, 0)


def test_a_call_sees_what_the_kernels_before_it_wrote(B):
    """Launches overlap the end of the kernel before them. Here that kernel writes the call's rows or
    its weights: another call (which lets its successor start early), a copy, a fill; on one stream
    and on two joined by events; eager, and captured and replayed. Each result has the bits that
    the same calls give when each waits for the one before."""
    d, f = 256, 264
    gen = torch.Generator().manual_seed(21)
    codes, scales = quantise(gen, d, d, 128)
    proj = B.QuantMatrix(codes.cuda(), scales.cuda(), d)
    up, down = rows(f, d, BF, 11, d ** -0.5), rows(d, f, BF, 12, f ** -0.5)
    w = dict(gate=torch.empty(f, d, dtype=BF, device="cuda"),
             up=torch.empty(f, d, dtype=BF, device="cuda"),
             down=torch.empty(d, f, dtype=BF, device="cuda"))
    target = B.DeviceFfn(dict(fmt="bf16", w_gate=w["gate"], w_up=w["up"], w_down=w["down"]), d, f)
    maker_g, _ = make(B, d, 520, seed=31)           # its rows become gate weights [f, d]
    maker_d, _ = make(B, f, 520, seed=32)           # ... down weights [d, f]
    mg, md = maker_g.descriptor(f), maker_d.descriptor(d)
    seeds_g = [rows(f, d, BF, 40 + i) for i in range(2)]
    seeds_d = [rows(d, f, BF, 50 + i) for i in range(2)]
    side = torch.cuda.Stream()
    descs = {T: (target.descriptor(T), proj.descriptor(T)) for T in (1, 4, 20)}
    big = target.descriptor(300)
    xs = {T: rows(T, d, BF, T) for T in (1, 4, 20, 300)}
    dy = rows(300, d, BF, 77)
    ws = B.alloc_ffn_workspace(big, backward=True)
    ws = torch.zeros(max(ws.numel(), *(B.ffn_workspace_size(D) for D in (mg, md)),
                         *(B.ffn_workspace_size(D[0]) for D in descs.values())),
                     dtype=torch.uint8, device="cuda")
    side_ws = torch.zeros_like(ws)

    def sequence(wait):
        out = []

        def call(fn, *a, **k):
            r = fn(*a, **k)
            wait()
            return r
        here = torch.cuda.current_stream()
        for i in (0, 1):
            call(w["up"].copy_, up)
            for T, (D, P) in descs.items():
                # gate weights, then down weights, from the call just before; down ones first
                call(B.ffn_forward, md, seeds_d[i], ws, out=w["down"])
                call(B.ffn_forward, mg, seeds_g[i], ws, out=w["gate"])
                y = call(B.ffn_forward, D, xs[T], ws)
                call(w["gate"].zero_)
                call(w["gate"].copy_, up)
                out.append(call(B.ffn_forward, D, y, ws))
                call(B.ffn_forward, md, seeds_d[1 - i], ws, out=w["down"])
                out.append(call(B.ffn_forward, D, out[-1], ws))
                z = call(B.matvec, P, out[-1], ws)
                out.append(call(B.matvec, P, z, ws))
                side.wait_stream(here)              # another stream's call in between
                with torch.cuda.stream(side):
                    z2 = call(B.matvec, P, out[-1], side_ws)
                here.wait_stream(side)
                out.append(call(B.ffn_forward, D, z2, ws))
                side.wait_stream(here)
            call(w["down"].copy_, down)
            pre = B.ffn_pre(big)
            y = call(B.ffn_forward, big, xs[300], ws, pre=pre)
            call(y.mul_, 0.5)
            out += [y, *call(B.ffn_backward, big, xs[300], dy, pre, ws)]
            call(pre.zero_)
            call(B.ffn_forward, mg, seeds_g[i], ws, out=w["gate"])
            y = call(B.ffn_forward, big, xs[300], ws, pre=pre)
            out += [y, *call(B.ffn_backward, big, xs[300], y, pre, ws)]
        return out
    want = [t.clone() for t in sequence(torch.cuda.synchronize)]
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(20):
        got = sequence(lambda: None)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sequence(lambda: None)
    for _ in range(20):
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i


def test_refusals(B):
    block, _ = make(B, 128, 128)
    int4, _ = make(B, 128, 128, fmt="int4")
    with pytest.raises(B.MoeError):
        int4.descriptor(33)
    d4 = int4.descriptor(4)
    with pytest.raises(B.MoeError):
        B.alloc_ffn_workspace(d4, backward=True)
    x = rows(4, 128, BF)
    with pytest.raises(B.MoeError):
        B.ffn_forward(d4, x, B.alloc_ffn_workspace(d4), pre=B.ffn_pre(d4))
    desc = block.descriptor(4)
    ws = B.alloc_ffn_workspace(desc)
    for call in (lambda p: B.ffn_backward(desc, x, x, p, ws),
                 lambda p: B.ffn_forward(desc, x, ws, pre=p)):
        with pytest.raises(B.MoeError):  # a forward workspace is too small for training calls
            call(B.ffn_pre(desc))
    for bad in (x.half(), x[:3], x.cpu(), rows(4, 256, BF)[:, ::2]):
        with pytest.raises(ValueError):
            B.ffn_forward(desc, bad, ws)
    with pytest.raises(B.MoeError):  # in place
        B.ffn_forward(desc, x, ws, out=x)
    with pytest.raises(ValueError):
        make(B, 132, 128)


def test_layer_block_and_projection_in_one_captured_step(B):
    """A decode step as a model runs it: the routed layer, a dense int4 block on its output, and
    the vocabulary projection, captured together; each stage against its own reference on the
    stage's actual input."""
    from expert_routed_ffn_route_b200 import synth
    T, V = 4, 1003
    cfg = synth.LayerConfig("run", T=T, d=256, E=16, k=2, f=128, fmt="int4", seed=3)
    L = synth.make_layer(cfg)
    dl = B.DeviceLayer(L)
    ld = dl.descriptor(T)
    lws = B.alloc_workspace(ld)
    block, W = make(B, 256, 512, fmt="int4")
    bd = block.descriptor(T)
    bws = B.alloc_ffn_workspace(bd)
    gen = torch.Generator().manual_seed(9)
    codes, scales = quantise(gen, V, 256, 64)
    proj = B.QuantMatrix(codes.cuda(), scales.cuda(), 256, 64)
    pd = proj.descriptor(T, y_dtype=F32)
    pws = B.alloc_matvec_workspace(pd)
    x = torch.from_numpy(L.x.view("int16")).cuda().view(BF)

    def step():
        a = B.layer_forward(ld, x, lws)
        b = B.ffn_forward(bd, a, bws)
        return a, b, B.matvec(pd, b, pws)
    eager = [t.clone() for t in step()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, eager):
        assert torch.equal(a, b)
    assert B.device_status(ld, lws) == 0
    ref, bound = ffn_ref(out[0], *W, "silu", BF)["y"]
    assert_close(out[1], ref, bound, BF, "block")
    ref, mag = matvec_ref(out[1].cpu(), dequantise(codes, scales, 64))
    assert_close(out[2], ref, mag * matvec_additions(256, 64) * 2.0 ** -23, F32, "projection")


@pytest.mark.parametrize("T", [1, 8])
def test_large_int4_block_with_large_scales(B, T):
    """Gate and up scales of 2^95 and more with rows around 2^-89: gates of ordinary size (2^14), in a
    block large enough for the products on shifted codes."""
    d, f = 2560, 4096
    gen = torch.Generator().manual_seed(13)
    bank, W = dict(fmt="int4", group=128, n_exp=1), []
    for m, N, K, by in (("gate", f, d, 2.0 ** 103), ("up", f, d, 2.0 ** 103), ("down", d, f, 1.0)):
        codes, scales = quantise(gen, N, K, 128)
        scales = (scales.double() * by).to(BF)
        bank["w_" + m], bank["s_" + m] = codes.cuda(), scales.cuda()
        W.append(dequantise(codes, scales, 128).cuda())
    x = 1 + torch.rand(T, d, generator=gen)
    x = (x * 2.0 ** -89 * (1 - 2 * torch.randint(0, 2, (T, d), generator=gen))).to(BF).cuda()
    desc = B.DeviceFfn(bank, d, f).descriptor(T)
    y = B.ffn_forward(desc, x, B.alloc_ffn_workspace(desc))
    assert torch.isfinite(y).all()
    ref, bound = ffn_ref(x, *W, "silu", BF)["y"]
    assert_close(y, ref, bound, BF, "y")
    assert_norm_close(y, ref, BF, "y")


def test_a_step_on_a_given_stream_keeps_to_its_memory(B):
    """As for the matrix: results of a step on another stream do not come from blocks that the
    current stream still reads, and its temporaries may be dropped at once."""
    T, d, f = 200, 1024, 2048
    block, _ = make(B, d, f)
    x, dy = rows(T, d, BF), rows(T, d, BF, seed=2)
    desc = block.descriptor(T)

    def step(stream):
        ws, pre = B.alloc_ffn_workspace(desc, backward=True), B.ffn_pre(desc)
        y = B.ffn_forward(desc, x, ws, pre=pre, stream=stream)
        return (y, *B.ffn_backward(desc, x, dy, pre, ws, stream=stream))
    want = [t.clone() for t in step(None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        blocks = [torch.full(t.shape, 5.0, dtype=BF, device="cuda") for t in want]
        ws, pre = B.alloc_ffn_workspace(desc, backward=True), B.ffn_pre(desc)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        torch.cuda._sleep(20_000_000)
        copies = [torch.empty_like(t).copy_(t) for t in blocks]
        del blocks
        y = B.ffn_forward(desc, x, ws, pre=pre, stream=side)
        got = (y, *B.ffn_backward(desc, x, dy, pre, ws, stream=side))
        n = ws.numel(), pre.shape
        del ws, pre
        junk = [torch.full((n[0],), 255, dtype=torch.uint8, device="cuda"),
                torch.full(n[1], 9.0, device="cuda")]
        torch.cuda.synchronize()
        assert all((c == 5).all() for c in copies) and len(junk) == 2
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            B.ffn_forward(desc, x, B.alloc_ffn_workspace(desc), stream=torch.cuda.Stream(device=1))


@pytest.mark.parametrize("fmt", [None, "int4"])
@pytest.mark.parametrize("T", [4, 20, 200])
def test_a_row_among_others(B, T, fmt):
    """At the same number of rows (up to 256, one row tile) a row's result, and its row of dx, have
    the same bits wherever it stands and whatever the others hold."""
    if fmt and T > 32:
        return
    block, _ = make(B, 256, 384, fmt=fmt)
    desc = block.descriptor(T)
    x, dy = rows(T, 256, BF, 31), rows(T, 256, BF, 32)
    x2, dy2 = rows(T, 256, BF, 33), rows(T, 256, BF, 34)
    x2[0], dy2[0] = x[T - 1], dy[T - 1]
    ws = B.alloc_ffn_workspace(desc)
    assert torch.equal(B.ffn_forward(desc, x, ws)[T - 1], B.ffn_forward(desc, x2, ws)[0])
    if not fmt:
        ws, pre, dx = B.alloc_ffn_workspace(desc, backward=True), B.ffn_pre(desc), []
        for a, b in ((x, dy), (x2, dy2)):
            B.ffn_forward(desc, a, ws, pre=pre)
            dx.append(B.ffn_backward(desc, a, b, pre, ws, need_dw=False)[0])
        assert torch.equal(dx[0][T - 1], dx[1][0])


@pytest.mark.parametrize("fmt,T", [("int4", 1), ("int4", 5), ("int4", 32), ("bf16", 3), ("bf16", 40)])
def test_a_block_is_a_layer_of_one_expert(B, fmt, T):
    """The two routes to a silu block agree: the routed layer with one expert and the block."""
    from types import SimpleNamespace
    d, f = 256, 384
    block, W = make(B, d, f, fmt="int4" if fmt == "int4" else None)
    bank = {k: v if isinstance(v, (str, int)) else v[None] for k, v in block.bank.items()}
    gate = torch.zeros(1, d, dtype=BF, device="cuda")
    dl = B.DeviceLayer.from_tensors(SimpleNamespace(d=d, f=f, E=1, k=1), gate, None, bank, None)
    ld, bd = dl.descriptor(T), block.descriptor(T)
    x = rows(T, d, BF, 41)
    ref, bound = ffn_ref(x, *W, "silu", BF)["y"]
    for y in (B.layer_forward(ld, x, B.alloc_workspace(ld)),
              B.ffn_forward(bd, x, B.alloc_ffn_workspace(bd))):
        assert_close(y, ref, bound, BF, fmt)
        assert_norm_close(y, ref, BF, fmt)
