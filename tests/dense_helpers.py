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
