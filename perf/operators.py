"""Cases, plain forms and calls of the dense operators beside the expert-routed layer.

Three operators of one dense feed-forward block and its projections:

matvec     y = x W^T (+ bias) for up to 32 rows x, W of 4-bit integers with a bf16 scale per
           group of 32, 64 or 128 values along K (the int4 bank encoding, one matrix)
ffn        y = Wd (act(Wg x) * (Wu x)): a dense gated feed-forward block, its weights bf16 or
           fp16 (any number of rows) or int4 with group scales (up to 32 rows)
ffn_train  the same block forward and backward: y, dx, dWg, dWu, dWd from x and dy

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LARGEST_FFN = 4096 * 2560 * 10240      # rows x d x f of the largest block
LARGEST_MATRIX = 131072 * 2560         # weights of the largest projection


def listed():
    return [
        # one decode token through a projection of the layer's own width: launch latency
        dict(name="matvec_token", op="matvec", T=1, N=1024, K=2560, group=128, x="bf16", y="bf16", bias=False),
        # one decode token onto a vocabulary, logits kept in fp32: streaming the weights
        dict(name="matvec_logits", op="matvec", T=1, N=131072, K=2560, group=128, x="bf16", y="fp32", bias=False),
        # a few draft tokens, an odd number of outputs, a bias, fp16, groups of 64
        dict(name="matvec_draft_odd", op="matvec", T=7, N=5003, K=4096, group=64, x="fp16", y="fp16", bias=True),
        # a verify batch over a long reduction, the finest groups
        dict(name="matvec_verify_g32", op="matvec", T=16, N=2560, K=10240, group=32, x="bf16", y="bf16", bias=False),
        # the largest row count of a verify chain
        dict(name="matvec_verify32", op="matvec", T=32, N=10240, K=2560, group=128, x="bf16", y="bf16", bias=False),
        # the dense block of one decode token at the shared expert's size, int4
        dict(name="ffn_int4_token", op="ffn", T=1, d=2560, f=1024, fmt="int4", act="silu"),
        # a wide dense block under a verify batch, int4
        dict(name="ffn_int4_verify", op="ffn", T=16, d=2560, f=10240, fmt="int4", act="gelu"),
        # the dense block of one decode token, bf16
        dict(name="ffn_token", op="ffn", T=1, d=2560, f=1024, fmt="bf16", act="silu"),
        # a ragged prompt chunk, fp16
        dict(name="ffn_prompt_ragged", op="ffn", T=509, d=2560, f=1024, fmt="fp16", act="silu"),
        # a long prompt through a wide dense block, bf16
        dict(name="ffn_long", op="ffn", T=4096, d=2560, f=10240, fmt="bf16", act="silu"),
        # a training step on a short ragged batch, widths that fill no tile
        dict(name="train_ragged", op="ffn_train", T=301, d=1032, f=2056, fmt="fp16", act="gelu"),
        # a training step on a long batch, the wide block
        dict(name="train_long", op="ffn_train", T=4096, d=2560, f=10240, fmt="bf16", act="silu"),
    ]


def _log(rng, lo, hi, step=1):
    """An integer in [lo, hi], uniform in its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "ffn", "ffn", "ffn_train"])
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        K = _log(rng, 512, 10240, group)
        N = min(_log(rng, 256, 131072), LARGEST_MATRIX // K)
        x = rng.choice(["bf16", "fp16"])
        return dict(op=op, T=rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 32)]), N=N, K=K, group=group,
                    x=x, y=rng.choice([x, "fp32"]), bias=rng.random() < 0.5)
    fmt = rng.choice(["bf16", "fp16", "int4"] if op == "ffn" else ["bf16", "fp16"])
    step = 128 if fmt == "int4" else 8
    d, f = _log(rng, 256, 4096, step), _log(rng, 256, 10240, step)
    few, most = (1, 32) if fmt == "int4" else (1, 4096) if op == "ffn" else (16, 4096)
    T = max(1, min(_log(rng, few, most), LARGEST_FFN // (d * f)))
    return dict(op=op, T=T, d=d, f=f, fmt=fmt, act=rng.choice(["silu", "gelu"]))


# ------------------------------------------------------------------ inputs


def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _quantise(gen, N, K, group, std):
    """N(0, std) weights as the banks hold them: codes int32 [N][K/8], scales bf16 [N][K/group]."""
    w = _normal(gen, N, K // group, group, std=std)
    s = (w.abs().amax(2) / 7).to(torch.bfloat16)
    q = torch.round(w / s.float()[..., None]).clamp_(-7, 7).to(torch.int32).view(N, K // 8, 8) & 15
    del w
    codes = q[..., 0].clone()
    for i in range(1, 8):
        codes |= q[..., i] << (4 * i)
    return codes, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "matvec":
        T, N, K, group = c["T"], c["N"], c["K"], c["group"]
        c["w"], c["s"] = _quantise(gen, N, K, group, K ** -0.5)
        c["rows"] = _normal(gen, T, K, dtype=DTYPES[c["x"]])
        c["b"] = _normal(gen, N, std=0.5) if c["bias"] else None
        if own:
            from expert_routed_ffn_route_b200 import binding as B
            c["matrix"] = B.QuantMatrix(c["w"], c["s"], K, group, bias=c["b"])
            c["desc"] = c["matrix"].descriptor(T, x_dtype=DTYPES[c["x"]], y_dtype=DTYPES[c["y"]])
            c["ws"] = B.alloc_matvec_workspace(c["desc"])
        return c
    T, d, f = c["T"], c["d"], c["f"]
    bank = c["bank"] = dict(fmt=c["fmt"], group=128, n_exp=1)
    for m, (N, K) in (("gate", (f, d)), ("up", (f, d)), ("down", (d, f))):
        if c["fmt"] == "int4":
            bank["w_" + m], bank["s_" + m] = _quantise(gen, N, K, 128, K ** -0.5)
        else:
            bank["w_" + m] = _normal(gen, N, K, std=K ** -0.5, dtype=DTYPES[c["fmt"]])
    t = torch.bfloat16 if c["fmt"] == "int4" else DTYPES[c["fmt"]]
    c["rows"] = _normal(gen, T, d, dtype=t)
    if c["op"] == "ffn_train":
        c["dy"] = _normal(gen, T, d, std=0.1, dtype=t)
    if own:
        from expert_routed_ffn_route_b200 import binding as B
        c["block"] = B.DeviceFfn(bank, d, f, act=c["act"])
        c["desc"] = c["block"].descriptor(T)
        c["ws"] = B.alloc_ffn_workspace(c["desc"], backward=c["op"] == "ffn_train")
    return c


# ------------------------------------------------------------------ one pass


def _dequantise(codes, scales, group):
    shifts = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    q = (codes[..., None] >> shifts) & 15
    q = q - ((q & 8) << 1)
    N = codes.shape[0]
    return (q.view(N, -1, group).float() * scales.float()[..., None]).view(N, -1)


def _weights(c):
    bank = c["bank"]
    if c["fmt"] == "int4":
        return [_dequantise(bank["w_" + m], bank["s_" + m], 128) for m in ("gate", "up", "down")]
    return [bank["w_" + m].float() for m in ("gate", "up", "down")]


ROOT_2_PI = math.sqrt(2 / math.pi)


def _activation(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    t = torch.tanh(ROOT_2_PI * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * ROOT_2_PI * (1 + 0.134145 * g * g)


def run(c):
    if own:
        from expert_routed_ffn_route_b200 import binding as B
        if c["op"] == "matvec":
            return B.matvec(c["desc"], c["rows"], c["ws"])
        if c["op"] == "ffn":
            return B.ffn_forward(c["desc"], c["rows"], c["ws"])
        pre = B.ffn_pre(c["desc"], device=c["rows"].device)
        y = B.ffn_forward(c["desc"], c["rows"], c["ws"], pre=pre)
        dx, dwg, dwu, dwd = B.ffn_backward(c["desc"], c["rows"], c["dy"], pre, c["ws"])
        return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
    x = c["rows"].float()
    if c["op"] == "matvec":
        y = x @ _dequantise(c["w"], c["s"], c["group"]).T
        if c["b"] is not None:
            y = y + c["b"]
        return y.to(DTYPES[c["y"]])
    wg, wu, wd = _weights(c)
    t = c["rows"].dtype
    g, u = x @ wg.T, x @ wu.T
    a, slope = _activation(g, c["act"])
    h = a * u
    y = (h @ wd.T).to(t)
    if c["op"] == "ffn":
        return y
    dy = c["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    return {"y": y, "dx": (dg @ wg + du @ wu).to(t), "dw_gate": (dg.T @ x).to(t), "dw_up": (du.T @ x).to(t),
            "dw_down": (dy.T @ h).to(t)}


# ------------------------------------------------------------------ floor and exact values


def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "matvec":
        T, N, K = c["T"], c["N"], c["K"]
        bytes_ = N * K // 2 + N * (K // c["group"]) * 2 + T * K * 2 + T * N * size[c["y"]] + (4 * N if c["bias"] else 0)
        return {"bytes": bytes_, "flops": 2 * T * N * K}
    T, d, f = c["T"], c["d"], c["f"]
    weights = 3 * d * f // 2 + 3 * d * f // 128 * 2 if c["fmt"] == "int4" else 3 * d * f * 2
    if c["op"] == "ffn":
        return {"bytes": weights + 2 * T * d * 2, "flops": 6 * T * d * f}
    # weights, x, dy in; y, dx and the weights' gradients out
    return {"bytes": 2 * weights + 4 * T * d * 2, "flops": 18 * T * d * f}


def _exact_matrix(codes, scales, group):
    """The weights in 64 bits, nibble by nibble: element 8 i + j of a row is bits 4 j .. 4 j + 3 of word i."""
    N, words = codes.shape
    w = torch.empty(N, words * 8, dtype=torch.float64, device=codes.device)
    for j in range(8):
        nibble = torch.bitwise_and(torch.bitwise_right_shift(codes, 4 * j), 15).to(torch.float64)
        w[:, j::8] = torch.where(nibble > 7, nibble - 16, nibble)
    return w * scales.to(torch.float64).repeat_interleave(group, dim=1)


def exact(case, seed):
    c = prepare(case, seed)
    x = c["rows"].to(torch.float64)
    if c["op"] == "matvec":
        y = torch.nn.functional.linear(x, _exact_matrix(c["w"], c["s"], c["group"]))
        return y if c["b"] is None else y + c["b"].to(torch.float64)
    bank = c["bank"]
    if c["fmt"] == "int4":
        ws = [_exact_matrix(bank["w_" + m], bank["s_" + m], 128) for m in ("gate", "up", "down")]
    else:
        ws = [bank["w_" + m].to(torch.float64) for m in ("gate", "up", "down")]
    linear, train = torch.nn.functional.linear, c["op"] == "ffn_train"
    for t in [x] + ws:
        t.requires_grad_(train)
    pre = linear(x, ws[0])
    a = torch.nn.functional.silu(pre) if c["act"] == "silu" else torch.nn.functional.gelu(pre, approximate="tanh")
    y = linear(a * linear(x, ws[1]), ws[2])
    if not train:
        return y
    dx, dwg, dwu, dwd = torch.autograd.grad(y, [x] + ws, c["dy"].to(torch.float64))
    return {"y": y.detach(), "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
