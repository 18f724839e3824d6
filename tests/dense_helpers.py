"""Plain implementations in 64 bits of the dense operators, and how far a result may be from
them.

Half a rounding step is eps / 2 relative to the value (bf16 2^-8, fp16 2^-11, fp32
2^-24). A sum of products in fp32 is off by at most (number of additions in a chain) * 2^-23 *
(sum of the terms' magnitudes): each addition rounds (2^-24), or truncates (2^-23) inside the
tensor core. Those magnitudes are computed here too, so every bound is an error bound, not a
fitted number.
"""
import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def quantise(gen, N, K, group, std=None):
    """Random weights in the int4 bank encoding: codes int32 [N, K/8], scales bf16 [N, K/group]."""
    w = torch.randn(N, K // group, group, generator=gen, dtype=torch.float32) * (std or K ** -0.5)
    s = (w.abs().amax(2) / 7).to(torch.bfloat16)
    q = torch.round(w / s.float()[..., None]).clamp_(-7, 7)
    q[0, 0, 0] = -8  # the one code the quantiser never gives
    return pack(q.reshape(N, K).to(torch.int64)), s


def pack(q):
    """Codes [N, K] (-8..7) -> int32 [N, K/8], element k in bits 4 (k mod 8) of word k/8."""
    n = (q & 15).view(q.shape[0], -1, 8)
    w = sum(n[..., j] << (4 * j) for j in range(8))
    return (w - ((w >> 31) << 32)).to(torch.int32)


def dequantise(codes, scales, group):
    q = torch.stack([(codes.to(torch.int64) >> (4 * j)) & 15 for j in range(8)], dim=2)
    q = (q - 16 * (q > 7)).reshape(codes.shape[0], -1).double()
    return q * scales.double().repeat_interleave(group, dim=1)


def matvec_ref(x, W, bias=None):
    """y and the sum of the terms' magnitudes, in 64 bits."""
    x = x.double()
    y, mag = x @ W.T, x.abs() @ W.abs().T
    return (y, mag) if bias is None else (y + bias.double(), mag + bias.double().abs())


def matvec_additions(K, group):
    """Additions one product of a row sees, at most: 8 tensor-core steps of 16 products in a
    128-wide slot (a step aligns and adds 17 terms: counted as 2), one per group, one per warp
    and per K part that brings a sum, the bias."""
    return 16 + K // group + 16 + 32 + 1


def assert_close(got, ref, bound, dtype, what=""):
    """|got - ref| within `bound` (before the result's own rounding) plus half a step of it."""
    got, ref = got.double().cpu(), ref.cpu()
    tol = bound.cpu() * (1 + HALF_STEP[dtype]) + HALF_STEP[dtype] * ref.abs() + TINY[dtype]
    bad = (got - ref).abs() - tol
    worst = bad.max().item() if bad.numel() else -1.0
    ratio = ((got - ref).abs() / tol).max().item() if bad.numel() else 0.0
    assert worst <= 0, f"{what}: {ratio:.3f} of the bound"
    return ratio


# ---------------------------------------------------------------------- dense gated block

ACT_LIPSCHITZ = 1.13   # max |act'| of silu (1.10) and gelu (1.13)
ACT2_LIPSCHITZ = 1.2   # max |act''| of silu (0.5) and tanh gelu (1.13)
FUNC = 2.0 ** -18      # relative error of the kernels' fp32 activations (fast exponential,
                       # |g| < 64: its argument's rounding, 64 * 2^-24 relative)


def activation(g, act):
    """act(g), act'(g) in the tensors' precision."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2 / torch.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def additions(K):
    """Additions of a K-long tensor-core product, at most: two per step of 16, and the partial
    sums of split products."""
    return K // 8 + 64


def ffn_ref(x, wg, wu, wd, act, dtype, dy=None, h_half=None):
    """{name: (value in 64 bits, bound of a kernel's error before the result's own rounding)}:
    fp32 sums, h, dg and du rounded to dtype (h with half steps of h_half), g and u kept in
    fp32."""
    half, tiny = HALF_STEP[dtype], TINY[dtype]
    h_half = half if h_half is None else h_half
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    T, d = x.shape
    f = wg.shape[0]
    u32 = 2.0 ** -23
    g, u = x @ wg.T, x @ wu.T
    eg = (x.abs() @ wg.abs().T) * additions(d) * u32
    eu = (x.abs() @ wu.abs().T) * additions(d) * u32
    a, da = activation(g, act)
    h = a * u
    ea = ACT_LIPSCHITZ * eg + FUNC * (a.abs() + g.abs())
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    eh = eh + h_half * (h.abs() + eh) + tiny
    out = {"y": (h @ wd.T, eh @ wd.abs().T + additions(f) * u32 * ((h.abs() + eh) @ wd.abs().T))}
    if dy is None:
        return out
    dy = dy.double()
    dh = dy @ wd
    edh = (dy.abs() @ wd.abs()) * additions(d) * u32
    dg, du = dh * u * da, dh * a
    eda = ACT2_LIPSCHITZ * eg + FUNC * (1 + g.abs())
    edg = edh * (u * da).abs() + dh.abs() * (eu * da.abs() + u.abs() * eda) + u32 * dg.abs()
    edu = edh * a.abs() + dh.abs() * ea + u32 * du.abs()
    edg = 1.01 * edg + half * (dg.abs() + edg) + tiny   # 1.01: the products of two errors
    edu = 1.01 * edu + half * (du.abs() + edu) + tiny
    mg, mu, mh = dg.abs() + edg, du.abs() + edu, h.abs() + eh
    out["dx"] = (dg @ wg + du @ wu, edg @ wg.abs() + edu @ wu.abs() +
                 additions(2 * f) * u32 * (mg @ wg.abs() + mu @ wu.abs()))
    n = additions(T) * u32
    out["dw_gate"] = (dg.T @ x, edg.T @ x.abs() + n * (mg.T @ x.abs()))
    out["dw_up"] = (du.T @ x, edu.T @ x.abs() + n * (mu.T @ x.abs()))
    out["dw_down"] = (dy.T @ h, dy.abs().T @ eh + n * (dy.abs().T @ mh))
    return out


def assert_norm_close(got, ref, dtype, what=""):
    """Relative error in the 2-norm: at most three roundings to dtype lie between the inputs and
    a result, each off by at most half a step of every value, independent of one another; a
    fourth is left for the fp32 sums. Catches a term that is missing or counted twice, which
    the worst-case bounds of long sums could hide."""
    got, ref = got.double(), ref.to(got.device)
    rel = ((got - ref).norm() / ref.norm().clamp_min(1e-300)).item()
    assert rel <= 4 * HALF_STEP[dtype], f"{what}: {rel:.3e}"
    return rel
