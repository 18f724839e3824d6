"""The 4-bit matrix-vector product on the GPU against a plain implementation in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
from dense_helpers import assert_close, dequantise, matvec_additions, matvec_ref, pack, quantise

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def B():
    from expert_routed_ffn_route_b200 import binding
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()
    return binding


def make(B, T, N, K, group, x_dtype=BF, y_dtype=None, bias=False, seed=0, **kw):
    gen = torch.Generator().manual_seed(seed)
    codes, scales = quantise(gen, N, K, group)
    b = torch.randn(N, generator=gen) if bias else None
    x = torch.randn(T, K, generator=gen).to(x_dtype)
    m = B.QuantMatrix(codes.cuda(), scales.cuda(), K, group, bias=None if b is None else b.cuda())
    desc = m.descriptor(T, x_dtype=x_dtype, y_dtype=y_dtype, **kw)
    return desc, x, dequantise(codes, scales, group), b


def check(y, x, W, b, group, what=""):
    ref, mag = matvec_ref(x, W, b)
    bound = mag * matvec_additions(W.shape[1], group) * 2.0 ** -23
    return assert_close(y, ref, bound, y.dtype, what)


SHAPES = [
    # T, N, K, group: one output, one group; ragged rows; K that ends inside a slot; K parts
    (1, 1, 32, 32), (1, 1, 128, 128), (1, 17, 64, 64), (2, 15, 96, 32), (3, 16, 192, 64),
    (1, 1000, 2560, 128), (5, 130, 1312, 32), (7, 333, 4160, 64), (8, 2560, 1024, 128),
    (9, 77, 640, 128), (16, 300, 1056, 32), (17, 33, 2560, 128), (32, 1000, 2560, 128),
    (32, 129, 10240, 32), (31, 65, 32768, 64), (1, 40, 32768, 128), (24, 2500, 768, 128),
    (1, 40000, 256, 128), (4, 20000, 384, 64),
]


@pytest.mark.parametrize("T,N,K,group", SHAPES)
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF, BF), (HF, F32), (BF, F32), (HF, HF)])
def test_matches_64_bits(B, T, N, K, group, x_dtype, y_dtype):
    desc, x, W, b = make(B, T, N, K, group, x_dtype, y_dtype, bias=(N % 2 == 1), seed=N + K)
    ws = B.alloc_matvec_workspace(desc)
    xd = x.cuda()
    y = B.matvec(desc, xd, ws)
    y2 = B.matvec(desc, xd, ws)  # the same workspace again: its counters are back at zero
    assert B.matvec_device_status(desc, ws) == (0, 0)
    assert y.dtype == y_dtype and tuple(y.shape) == (T, N)
    assert torch.equal(y, y2)
    check(y, x, W, b, group, f"{T}x{N}x{K} g{group}")


def test_many_outputs_with_k_in_parts(B):
    """More row tiles than a workspace has fixed counters for, K split: the call clears its own,
    whatever the workspace held there."""
    T, N, K = 32, 131120, 4096
    gen = torch.Generator().manual_seed(8)
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=gen).to(torch.int32)
    scales = (torch.rand(N, K // 128, generator=gen) * 2.0 ** -8 + 2.0 ** -9).to(BF)
    x = torch.randn(T, K, generator=gen).to(BF)
    m = B.QuantMatrix(codes.cuda(), scales.cuda(), K)
    desc = m.descriptor(T, y_dtype=F32)
    ws = B.alloc_matvec_workspace(desc)
    assert ws.numel() > 256 + 4 * 8192 + 4 * (N // 16)      # split
    y = B.matvec(desc, x.cuda(), ws)
    ws[256 + 4 * 8192:] = 255
    assert torch.equal(y, B.matvec(desc, x.cuda(), ws))
    assert torch.equal(y, B.matvec(desc, x.cuda(), ws))
    for at in (0, N // 2, N - 3000):                        # three stretches against 64 bits
        rows = slice(at, at + 3000)
        check(y[:, rows], x, dequantise(codes[rows], scales[rows], 128), None, 128, at)


def test_a_matrix_beyond_32_bits(B):
    """Codes of more than 2^32 bytes."""
    N, K = 600_011, 16384
    gen = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=gen, device="cuda",
                          dtype=torch.int32)
    scales = (torch.rand(N, K // 64, generator=gen, device="cuda") * 2.0 ** -8 + 2.0 ** -9).to(BF)
    m = B.QuantMatrix(codes, scales, K, 64)
    for T in (1, 8):
        x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(BF)
        desc = m.descriptor(T, y_dtype=F32)
        y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
        for at in (0, 2 ** 32 // (K // 2) - 100, N - 500):
            part = slice(at, at + 500)
            W = dequantise(codes[part].cpu(), scales[part].cpu(), 64)
            check(y[:, part], x, W, None, 64, f"{T} rows, from {at}")


def test_rows_far_apart(B):
    """Rows of x and y 2^30 elements apart, the last beyond 2^32 bytes."""
    T, N, K, ld = 4, 1000, 640, 1 << 30
    desc, x, W, b = make(B, T, N, K, 128, ldx=ld, ldy=ld)
    xb = torch.empty((T - 1) * ld + K, dtype=BF, device="cuda").as_strided((T, K), (ld, 1))
    yb = torch.empty((T - 1) * ld + N, dtype=BF, device="cuda").as_strided((T, N), (ld, 1))
    xb.copy_(x)
    check(B.matvec(desc, xb, B.alloc_matvec_workspace(desc), out=yb), x, W, b, 128)


# ---- calls large enough for the products on shifted codes (few rows, groups of 128): the sums
# are sum((q + 8) x) - 8 sum(x), so their terms' magnitudes are those of |q| + 8

BIG = (40000, 640)  # N, K: an odd number of groups


def check_shifted(y, x, W, scales, what=""):
    ref, _ = matvec_ref(x, W)
    W8 = W.abs() + 8 * scales.double().repeat_interleave(128, 1)
    bound = (x.double().abs() @ W8.T) * matvec_additions(W.shape[1], 128) * 2.0 ** -23
    return assert_close(y, ref, bound, y.dtype, what)


@pytest.fixture(scope="module")
def big(B):
    gen = torch.Generator().manual_seed(11)
    N, K = BIG
    codes, scales = quantise(gen, N, K, 128)
    codes[5] = 0                                    # a row of zero codes
    return B.QuantMatrix(codes.cuda(), scales.cuda(), K), dequantise(codes, scales, 128), scales


@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF, F32), (HF, F32), (BF, BF), (HF, HF)])
def test_large_matrix_few_rows(B, big, T, x_dtype, y_dtype):
    m, W, scales = big
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, BIG[1], generator=gen).to(x_dtype)
    desc = m.descriptor(T, x_dtype=x_dtype, y_dtype=y_dtype)
    ws = B.alloc_matvec_workspace(desc)
    y = B.matvec(desc, x.cuda(), ws)
    assert torch.equal(y, B.matvec(desc, x.cuda(), ws))
    check_shifted(y, x, W, scales)
    assert B.matvec_device_status(desc, ws) == (0, 0)


@pytest.mark.parametrize("value", [2.0 ** 25, 2.0 ** 26, 2.0 ** 100, 2.0 ** -90, 2.0 ** -91, 2.0 ** -120,
                                   2.0 ** -133])
def test_large_matrix_magnitudes_at_the_ends_of_the_range(B, big, value):
    """Rows whose bf16 magnitudes reach the ends of the shifted form's range, and leave it."""
    m, W, scales = big
    x = torch.zeros(1, BIG[1], dtype=BF)
    x[0, ::3] = value
    x[0, 1::6] = -value
    desc = m.descriptor(1, y_dtype=F32)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
    check_shifted(y, x, W, scales)
    # beside ordinary values: a term of every size counts
    x2 = x.clone()
    x2[0, 2] = 1.0
    y = B.matvec(desc, x2.cuda(), B.alloc_matvec_workspace(desc))
    check_shifted(y, x2, W, scales)


@pytest.mark.parametrize("x_dtype", [BF, HF])
def test_large_matrix_infinities_and_nan(B, big, x_dtype):
    m, W, scales = big
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(3, BIG[1], generator=gen).to(x_dtype)
    x[1, 300], x[2, 7] = float("inf"), float("nan")
    desc = m.descriptor(3, x_dtype=x_dtype, y_dtype=F32)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc)).cpu()
    check_shifted(y[:1], x[:1], W, scales)
    w = W[:, 300]
    assert torch.isnan(y[1][w == 0]).all() and torch.isnan(y[2]).all()
    assert torch.equal(y[1][w != 0].double(), torch.sign(w[w != 0]) * float("inf"))


@pytest.mark.parametrize("x_dtype", [BF, HF])
def test_large_matrix_single_weights(B, big, x_dtype):
    """One-hot rows through the shifted form are exact too: both terms are small integers times
    the one activation."""
    m, W, _ = big
    for k0 in (0, 121, 256, 632):
        x = torch.zeros(8, BIG[1], dtype=x_dtype)
        x[torch.arange(8), k0 + torch.arange(8)] = -0.75
        desc = m.descriptor(8, x_dtype=x_dtype, y_dtype=F32)
        y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
        assert torch.equal(y.cpu().double(), -0.75 * W[:, k0:k0 + 8].T), k0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_dtype", [BF, HF])
def test_every_code_and_position_is_exact(B, group, x_dtype):
    """One-hot rows pick single weights out: the result is that code times its scale, exactly
    (products of 4 and 8 significant bits), wherever in the row it stands."""
    K, N = 2 * group + 128 if group != 32 else 416, 16
    q = torch.arange(N * K).view(N, K) * 7 % 16 - 8
    scales = torch.tensor([2.0 ** (i % 5 - 2) for i in range(N * (K // group))]).view(N, -1).to(BF)
    m = B.QuantMatrix(pack(q).cuda(), scales.cuda(), K, group)
    W = dequantise(pack(q), scales, group)
    assert torch.equal(W, q.double() * scales.double().repeat_interleave(group, 1))
    for k0 in range(0, K, 32):
        x = torch.zeros(32, K, dtype=x_dtype)
        x[torch.arange(32), k0 + torch.arange(32)] = 1.5
        desc = m.descriptor(32, x_dtype=x_dtype, y_dtype=F32)
        y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
        assert torch.equal(y.cpu().double(), 1.5 * W[:, k0:k0 + 32].T), k0


def test_strided_rows_and_what_lies_between_them(B):
    T, N, K = 6, 50, 256
    desc, x, W, b = make(B, T, N, K, 128, ldx=K + 24, ldy=N + 13, bias=True)
    xb = torch.full((T, K + 24), float("nan"), dtype=BF, device="cuda")
    xb[:, :K] = x.cuda()
    yb = torch.full((T + 1, N + 13), 7.0, dtype=BF, device="cuda")
    B.matvec(desc, xb[:, :K], B.alloc_matvec_workspace(desc), out=yb[:T, :N])
    check(yb[:T, :N], x, W, b, 128)
    assert (yb[:, N:] == 7).all() and (yb[T:] == 7).all()
    # the output made by the call has the descriptor's row distance
    y = B.matvec(desc, xb[:, :K], B.alloc_matvec_workspace(desc))
    assert y.stride(0) == N + 13 and torch.equal(y, yb[:T, :N])


@pytest.mark.parametrize("T", [1, 9, 32])
def test_infinities_and_nan_stay_in_their_rows(B, T):
    """An infinite or NaN activation reaches its own row only, with the signs of the codes."""
    N, K = 64, 512
    desc, x, W, b = make(B, T, N, K, 128, y_dtype=F32)
    x[T - 1, 300] = float("inf")
    ws = B.alloc_matvec_workspace(desc)
    y = B.matvec(desc, x.cuda(), ws).cpu()
    expect = torch.where(W[:, 300] == 0, torch.tensor(float("nan"), dtype=torch.float64),
                         torch.sign(W[:, 300]) * float("inf"))
    assert torch.equal(torch.isnan(y[T - 1]), torch.isnan(expect))
    ok = ~torch.isnan(expect)
    assert torch.equal(y[T - 1].double()[ok], expect[ok])
    x[T - 1, 300] = float("nan")
    y = B.matvec(desc, x.cuda(), ws).cpu()
    assert torch.isnan(y[T - 1]).all()
    if T > 1:
        check(y[:T - 1], x[:T - 1], W, b, 128)


def test_large_activations_overflow_only_where_the_result_does(B):
    """Codes enter the products without an offset: activations near the end of bf16's range
    do not overflow where codes of both signs cancel."""
    K, N = 256, 16
    q = torch.ones(N, K, dtype=torch.int64)
    q[:, 1::2] = -1
    m = B.QuantMatrix(pack(q).cuda(), torch.ones(N, K // 128, dtype=BF).cuda(), K, 128)
    desc = m.descriptor(1, y_dtype=F32)
    x = torch.full((1, K), 2.0 ** 120, dtype=BF)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
    assert (y == 0).all()


@pytest.mark.parametrize("T,N,K,group", [(1, 65536, 2560, 128), (8, 30000, 4096, 64),
                                         (16, 20000, 2560, 32), (32, 16384, 10240, 128)])
def test_large_calls_repeat_bit_for_bit(B, T, N, K, group):
    desc, x, W, b = make(B, T, N, K, group, y_dtype=F32)
    ws, xd = B.alloc_matvec_workspace(desc), x.cuda()
    first = B.matvec(desc, xd, ws)
    for _ in range(100):
        again = [B.matvec(desc, xd, ws) for _ in range(5)][-1]
        assert torch.equal(again, first)


@pytest.mark.parametrize("T,K", [(1, 2560), (32, 10240)])
def test_captured_replayed_and_on_another_stream(B, T, K):
    """Two captured graphs with a workspace each, replayed at once on two streams."""
    N = 777
    calls = []
    for seed in (1, 2):
        desc, x, W, b = make(B, T, N, K, 128, seed=seed)
        calls.append(dict(desc=desc, x=x.cuda(), xc=x, W=W, ws=B.alloc_matvec_workspace(desc),
                          y=torch.empty(T, N, dtype=BF, device="cuda"), g=torch.cuda.CUDAGraph(),
                          s=torch.cuda.Stream()))
        B.matvec(desc, calls[-1]["x"], calls[-1]["ws"], out=calls[-1]["y"])
    torch.cuda.synchronize()
    for c in calls:
        with torch.cuda.graph(c["g"], stream=c["s"]):
            B.matvec(c["desc"], c["x"], c["ws"], out=c["y"])
        c["y"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            with torch.cuda.stream(c["s"]):
                c["g"].replay()
    torch.cuda.synchronize()
    for c in calls:
        check(c["y"], c["xc"], c["W"], None, 128)
        s = torch.cuda.Stream()
        y = B.matvec(c["desc"], c["x"], c["ws"], stream=s)
        s.synchronize()
        assert torch.equal(y, c["y"])


def test_a_row_comes_out_the_same_whatever_the_others_hold(B):
    T, N, K = 8, 96, 1280
    desc, x, W, b = make(B, T, N, K, 128)
    ws = B.alloc_matvec_workspace(desc)
    y = B.matvec(desc, x.cuda(), ws)
    x2 = torch.randn(T, K).to(BF)
    x2[3] = x[5]
    y2 = B.matvec(desc, x2.cuda(), ws)
    assert torch.equal(y2[3], y[5])


def test_same_encoding_as_an_expert_bank(B):
    """A projection of an int4 expert bank, taken as one matrix, equals the bank's own
    dequantised product."""
    from expert_routed_ffn_route_b200 import synth
    from oracle import moe_oracle as O
    cfg = synth.LayerConfig("mv", T=3, d=256, E=4, k=2, f=128, fmt="int4", seed=5)
    L = synth.make_layer(cfg)
    dl = B.DeviceLayer(L)
    bank = dl.banks["routed"]
    m = B.QuantMatrix(bank["w_down"][2], bank["s_down"][2], cfg.f)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(3, cfg.f, generator=gen).to(BF)
    desc = m.descriptor(3, y_dtype=F32)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
    arrays = L.routed.arrays()
    W = dequantise(torch.from_numpy(arrays["w_down"][2].view("int32")),
                   torch.from_numpy(arrays["s_down"][2].view("int16")).view(BF), 128)
    assert W.shape == (cfg.d, cfg.f) and O is not None
    check(y, x, W, None, 128)


@pytest.mark.parametrize("x_dtype,scale,value", [
    (BF, 2.0 ** 94, 2.0 ** -40), (BF, 2.0 ** 95, 2.0 ** -60), (BF, 2.0 ** 127, 2.0 ** -85),
    (BF, 2.0 ** -126, 2.0 ** 20), (BF, 2.0 ** -133, 2.0 ** 24),
    (HF, 2.0 ** 103, 2.0 ** -8), (HF, 2.0 ** 104, 2.0 ** -12), (HF, 2.0 ** 127, 2.0 ** -14),
    (HF, 2.0 ** -126, 2.0 ** 12)])
@pytest.mark.parametrize("T", [1, 8])
def test_large_matrix_scales_at_the_ends_of_their_type(B, big, T, x_dtype, scale, value):
    """Scales up to bf16's largest binade and down to its subnormals, beside rows (inside the
    shifted form's range) that bring the results back to fp32's: every result is finite and as
    exact as with ordinary scales."""
    m, _, scales = big
    codes, (N, K) = m.codes.cpu(), BIG
    s = (torch.frexp(scales.float())[0].double() * 2 * scale).to(BF)   # [1, 2) times scale
    assert torch.isfinite(s).all()
    gen = torch.Generator().manual_seed(12)
    x = 1 + torch.rand(T, K, generator=gen)
    x = (x * value * (1 - 2 * torch.randint(0, 2, (T, K), generator=gen))).to(x_dtype)
    desc = B.QuantMatrix(m.codes, s.cuda(), K).descriptor(T, x_dtype=x_dtype, y_dtype=F32)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
    assert torch.isfinite(y).all()
    check_shifted(y, x, dequantise(codes, s, 128), s)


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("K,group", [(32, 32), (416, 32), (192, 64), (320, 64)])
def test_an_infinite_scale_of_the_last_group(B, T, K, group):
    """K that ends inside a unit of 128: what lies behind the last group takes no part, its scale's
    infinity neither (it would meet a sum of zero)."""
    N = 40
    gen = torch.Generator().manual_seed(K)
    q = torch.randint(1, 8, (N, K), generator=gen)
    scales = torch.full((N, K // group), 0.5).to(BF)
    scales[::2, -1] = float("inf")
    x = (torch.rand(T, K, generator=gen) + 0.5).to(BF)
    desc = B.QuantMatrix(pack(q).cuda(), scales.cuda(), K, group).descriptor(T, y_dtype=F32)
    y = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc)).cpu()
    assert (y[:, ::2] == float("inf")).all()
    check(y[:, 1::2], x, dequantise(pack(q)[1::2], scales[1::2], group), None, group)


def test_calls_on_a_given_stream_keep_to_their_memory(B):
    """Blocks that the current stream has freed but whose readers are still queued there are not
    handed out as results on another stream, and what a call on another stream uses is not handed
    out again, when freed at once, before that call has run."""
    T, N, K = 32, 8192, 2560
    desc, x, W, b = make(B, T, N, K, 128)
    want = B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc))
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(here)
        torch.cuda.synchronize()
        # a reader of a freed block queued here, behind a pause
        block = torch.full((T, N), 5.0, dtype=BF, device="cuda")
        xd, ws = x.cuda(), B.alloc_matvec_workspace(desc)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        copy = torch.empty_like(block).copy_(block)
        del block
        y = B.matvec(desc, xd, ws, stream=side)
        torch.cuda.synchronize()
        assert (copy == 5).all() and torch.equal(y, want)
        # the call's own tensors, freed while it waits behind a pause on its stream
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y = B.matvec(desc, xd, ws, stream=side)
        shape = xd.shape, ws.shape
        del xd, ws
        junk = [torch.full(shape[0], 9.0, dtype=BF, device="cuda") for _ in range(4)]
        junk += [torch.full(shape[1], 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(y, want) and B.matvec_device_status(desc, junk[-1].zero_()) == (0, 0)


@pytest.mark.parametrize("T", [1, 2, 8, 32])
def test_rows_and_results_in_one_array(B, T):
    """x and y as columns of one array: neither touches the other or what lies beside them."""
    N, K, ld = 500, 1280, 2560
    desc, x, W, b = make(B, T, N, K, 128, ldx=ld, ldy=ld)
    buf = torch.full((T, ld), 3.0, dtype=BF, device="cuda")
    buf[:, 512:512 + K] = x.cuda()
    for at in (0, 12, 512 + K, ld - N):
        buf[:, at:at + N] = 7.0
        B.matvec(desc, buf[:, 512:512 + K], B.alloc_matvec_workspace(desc), out=buf[:, at:at + N])
        check(buf[:, at:at + N], x, W, b, 128, at)
        assert torch.equal(buf[:, 512:512 + K].cpu(), x)
        buf[:, at:at + N] = 3.0
        assert (buf[:, :512] == 3).all() and (buf[:, 512 + K:] == 3).all()
    if T > 1:
        with pytest.raises(B.MoeError):
            B.matvec(desc, buf[:, 512:512 + K], B.alloc_matvec_workspace(desc), out=buf[:, 13:13 + N])


def test_an_experts_matrices_as_the_oracle_reads_them(B):
    """The three matrices of one expert of an int4 bank, as products against the oracle's
    dequantised weights, and as a dense block against the oracle's expert."""
    import numpy as np
    from dense_helpers import assert_norm_close, ffn_ref
    from expert_routed_ffn_route_b200 import synth
    from oracle import moe_oracle as O
    cfg = synth.LayerConfig("mv", T=3, d=256, E=4, k=2, f=384, fmt="int4", seed=6)
    L = synth.make_layer(cfg)
    dl, arrays, e = B.DeviceLayer(L), L.routed.arrays(), 1
    bank, W = dl.banks["routed"], []
    gen = torch.Generator().manual_seed(3)
    for m, N, K in (("gate", cfg.f, cfg.d), ("up", cfg.f, cfg.d), ("down", cfg.d, cfg.f)):
        W.append(O.dequantize(arrays["w_" + m][e], arrays["s_" + m][e], "int4", 128, K))
        assert W[-1].shape == (N, K)
        x = torch.randn(3, K, generator=gen).to(BF)
        desc = B.QuantMatrix(bank["w_" + m][e], bank["s_" + m][e], K).descriptor(3, y_dtype=F32)
        check(B.matvec(desc, x.cuda(), B.alloc_matvec_workspace(desc)), x, torch.from_numpy(W[-1]),
              None, 128, m)
    block = B.DeviceFfn({k: v if isinstance(v, (str, int)) else v[e] for k, v in bank.items()
                         if k != "n_exp"}, cfg.d, cfg.f)
    x = torch.randn(3, cfg.d, generator=gen).to(BF)
    desc = block.descriptor(3)
    y = B.ffn_forward(desc, x.cuda(), B.alloc_ffn_workspace(desc))
    want = torch.from_numpy(O.expert_ffn(x.double().numpy(), *W))
    bound = ffn_ref(x, *(torch.from_numpy(w) for w in W), "silu", BF)["y"][1]
    assert np.isfinite(want.numpy()).all()
    assert_close(y, want, bound, BF, "block")
    assert_norm_close(y, want, BF, "block")


@pytest.mark.parametrize("x_dtype", [BF, HF])
def test_large_matrix_a_row_among_ordinary_rows(B, big, x_dtype):
    """In the shifted form too, at the same number of rows, a row has the same bits whatever
    ordinary values the others hold; beside a NaN (the other form) it is within the bound."""
    m, W, scales = big
    gen = torch.Generator().manual_seed(21)
    x = torch.randn(8, BIG[1], generator=gen).to(x_dtype)
    desc = m.descriptor(8, x_dtype=x_dtype, y_dtype=F32)
    ws = B.alloc_matvec_workspace(desc)
    y = B.matvec(desc, x.cuda(), ws)
    other = torch.randn(8, BIG[1], generator=gen).to(x_dtype)
    other[2] = x[6]
    assert torch.equal(B.matvec(desc, other.cuda(), ws)[2], y[6])
    other[5, 17] = float("nan")
    z = B.matvec(desc, other.cuda(), ws)
    assert torch.isnan(z[5]).all()
    check_shifted(z[2:3], x[6:7], W, scales)


def test_a_result_of_another_stream_dropped_while_it_is_read(B):
    """A result that work queued here still reads is not overwritten by the next call on the stream
    that made it; eager, and with the call on a captured side stream."""
    T, N, K = 32, 8192, 2560
    desc, x, W, b = make(B, T, N, K, 128)
    ws, xd = B.alloc_matvec_workspace(desc), x.cuda()
    want = B.matvec(desc, xd, ws)
    side, zero = torch.cuda.Stream(), torch.zeros_like(xd)
    torch.cuda.synchronize()
    for _ in range(3):
        y = B.matvec(desc, xd, ws, stream=side)
        side.synchronize()
        torch.cuda._sleep(20_000_000)
        copy = y.clone()
        del y
        junk = [B.matvec(desc, zero, ws, stream=side) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want) and all((j == 0).all() for j in junk)
    g, here = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=here):
        side.wait_stream(here)
        t = xd + 0
        y = B.matvec(desc, t, ws, stream=side)
        del t
        here.wait_stream(side)
        z = y + 0
        y2 = B.matvec(desc, xd, ws, stream=here)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want) and torch.equal(y2, want)


def test_many_outputs_captured_and_replayed(B):
    """The call that clears its own counters first, in a graph, twice in a row and over a workspace
    that another call has filled in between."""
    T, N, K = 32, 131120, 4096
    gen = torch.Generator().manual_seed(8)
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=gen).to(torch.int32).cuda()
    scales = (torch.rand(N, K // 128, generator=gen) * 2.0 ** -8 + 2.0 ** -9).to(BF).cuda()
    m = B.QuantMatrix(codes, scales, K)
    desc, few = m.descriptor(T), m.descriptor(9)
    ws = torch.zeros(max(B.matvec_workspace_size(d) for d in (desc, few)), dtype=torch.uint8,
                     device="cuda")
    x = torch.randn(T, K, generator=gen).to(BF).cuda()
    want, want9 = B.matvec(desc, x, ws), B.matvec(few, x[:9], ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [B.matvec(desc, x, ws), B.matvec(desc, x, ws), B.matvec(few, x[:9], ws),
               B.matvec(desc, x, ws)]
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want9 if len(y) == 9 else want) for y in out)
    assert B.matvec_device_status(desc, ws) == (0, 0)


def test_two_host_threads_at_once(B):
    """Calls from two threads, each with its stream and workspace."""
    import threading
    jobs, errors = [], []
    for seed in (1, 2):
        desc, x, W, b = make(B, 16, 2560, 10240, 32, seed=seed)
        jobs.append((desc, x.cuda(), B.alloc_matvec_workspace(desc), torch.cuda.Stream()))
    want = [B.matvec(desc, x, ws) for desc, x, ws, _ in jobs]
    torch.cuda.synchronize()

    def work(i):
        try:
            desc, x, ws, s = jobs[i]
            with torch.cuda.stream(s):
                for _ in range(200):
                    y = B.matvec(desc, x, ws)
                s.synchronize()
                assert torch.equal(y, want[i])
        except BaseException as e:  # noqa: BLE001 (reported by the main thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
