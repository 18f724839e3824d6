"""Host-side checks of the dense operators' entry points and of their binding (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from expert_routed_ffn_route_b200 import _build, binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned non-NULL stand-in: validation never dereferences


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


def matrix(**kw):
    m = binding.MoeMatrix(8, 1000, 2560, 128, 0, 0, 2560, 1000, FAKE, FAKE, None)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("fields,code", [
    ({}, 0), ({"group": 64}, 0), ({"group": 32, "K": 2592, "ldx": 2592}, 0), ({"y_type": 2}, 0),
    ({"x_type": 1, "y_type": 1}, 0), ({"bias": FAKE}, 0), ({"T": 32}, 0), ({"ldy": 1003}, 0),
    ({"T": 0}, -1), ({"N": 0}, -1), ({"K": 0}, -1), ({"K": -128}, -1), ({"T": 33}, -2),
    ({"group": 16}, -1), ({"group": 0}, -1), ({"K": 2592, "ldx": 2592}, -1),
    ({"K": 32768 + 128, "ldx": 40000}, -2), ({"N": (1 << 24) + 1, "ldy": 1 << 25}, -2),
    ({"x_type": 2}, -1), ({"x_type": 3}, -1), ({"y_type": 1}, -1), ({"y_type": -1}, -1),
    ({"ldx": 2552}, -1), ({"ldx": 2564}, -1), ({"ldy": 999}, -1), ({"ldx": 1 << 41}, -2),
    ({"w": None}, -1), ({"w": FAKE + 8}, -1), ({"s": None}, -1), ({"s": FAKE + 1}, -1),
    ({"bias": FAKE + 2}, -1),
])
def test_matvec_validation(lib, fields, code):
    m = matrix(**fields)
    assert lib.moe_matvec_validate(ctypes.byref(m)) == code
    size = lib.moe_matvec_workspace_size(ctypes.byref(m))
    assert (size >= 256 and size % 256 == 0) if code == 0 else size == 0


def test_matvec_rejects_bad_arguments_before_any_cuda_call(lib):
    m = matrix()
    call = lambda x, y, ws, n: lib.moe_matvec(ctypes.byref(m), x, y, ws, n, None)  # noqa: E731
    far = 1 << 40
    m.w, m.s = 1 << 41, 1 << 42
    assert call(None, far, FAKE, 1 << 30) == -1
    assert call(FAKE, None, FAKE, 1 << 30) == -1
    assert call(FAKE + 2, far, FAKE, 1 << 30) == -1
    assert call(FAKE, far + 1, FAKE, 1 << 30) == -1
    assert call(FAKE, far, None, 1 << 30) == -5
    assert call(FAKE, far, FAKE + 16, 1 << 30) == -5
    assert call(FAKE, far, FAKE, 128) == -5
    assert call(FAKE, FAKE + 64, FAKE, 1 << 30) == -1      # y over x
    assert call(FAKE, m.w + 64, FAKE, 1 << 30) == -1       # y over the codes
    assert call(FAKE, m.s + 64, FAKE, 1 << 30) == -1       # y over the scales
    assert call(FAKE, far, far, 1 << 30) == -1             # y over the workspace
    assert lib.moe_matvec(None, FAKE, far, FAKE, 1 << 30, None) == -1


def test_matvec_splits_long_rows_into_parts_with_workspace(lib):
    """Rows that fit shared memory need no partial sums; longer ones keep one per part."""
    small = lib.moe_matvec_workspace_size(ctypes.byref(matrix(T=1)))
    long = lib.moe_matvec_workspace_size(ctypes.byref(matrix(T=32, K=32768, ldx=32768)))
    assert small == 256 and long > 1000 * 32 * 4


def test_struct_layouts_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "abi.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_b200.h"\n'
                   'int main(void) { printf("%zu %zu %zu\\n", sizeof(moe_matrix),'
                   ' offsetof(moe_matrix, ldx), offsetof(moe_matrix, bias)); return 0; }\n')
    exe = tmp_path / "abi"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                            check=True).stdout.split()]
    M = binding.MoeMatrix
    assert sizes == [ctypes.sizeof(M), M.ldx.offset, M.bias.offset]


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    codes = torch.zeros(4, 16, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.QuantMatrix(codes, torch.zeros(4, 1, dtype=torch.bfloat16), 128)  # not on a GPU
    with pytest.raises(ValueError):
        binding.QuantMatrix(codes, torch.zeros(4, 1, dtype=torch.bfloat16), 130)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    check = lambda t, stride=None: binding._check_rows(  # noqa: E731 (-1: the CPU's index)
        t, "x", (4, 8), torch.bfloat16, -1, stride)
    check(x)
    wide = torch.zeros(4, 24, dtype=torch.bfloat16)
    check(wide[:, :8], 24)
    for t in (wide[:, :8], wide[:, ::3], x.T, x.float(), x[:3], x[:1].expand(4, 8), x[None]):
        with pytest.raises(ValueError):
            check(t)
    with pytest.raises(ValueError):
        check(x, 24)
    with pytest.raises(ValueError):
        binding._check_rows(x, "x", (4, 8), torch.bfloat16, 0)


def ffn(fmt=16, **kw):
    bank = binding.MoeBank(fmt, 128, 1, 0, *([FAKE] * 6), None, None, None)
    F = binding.MoeFfn(40, 2560, 1024, 0, bank)
    for k, v in kw.items():
        setattr(F.bank if k.startswith("w_") or k.startswith("s_") or
                k in ("fmt", "group", "n_exp") else F, k, v)
    return F


@pytest.mark.parametrize("fields,code", [
    ({}, 0), ({"fmt": 17}, 0), ({"act": 1}, 0), ({"d": 8, "f": 8}, 0), ({"T": 1}, 0),
    ({"fmt": 4, "T": 32}, 0), ({"s_gate": None, "s_up": None, "s_down": None}, 0),
    ({"T": 1 << 20, "d": 32768, "f": 32768}, 0),
    ({"T": 0}, -1), ({"T": (1 << 20) + 1}, -2), ({"d": 4}, -1), ({"d": 12}, -1), ({"f": 0}, -1),
    ({"d": 32776}, -2), ({"f": 40000}, -2), ({"act": 2}, -1), ({"n_exp": 2}, -1), ({"n_exp": 0}, -1),
    ({"fmt": 4, "T": 33}, -2), ({"fmt": 4, "T": 4, "d": 192}, -1),
    ({"fmt": 4, "T": 4, "group": 64}, -1), ({"fmt": 4, "T": 4, "s_up": None}, -1),
    ({"fmt": 8}, -2), ({"fmt": 41}, -2), ({"fmt": 3}, -1), ({"w_up": None}, -1),
    ({"w_down": FAKE + 8}, -1),
])
def test_ffn_validation(lib, fields, code):
    F = ffn(**fields)
    assert lib.moe_ffn_validate(ctypes.byref(F)) == code
    fwd = lib.moe_ffn_workspace_size(ctypes.byref(F), 0)
    both = lib.moe_ffn_workspace_size(ctypes.byref(F), 1)
    if code == 0:
        assert fwd >= 256 + 2 * F.T * F.f and fwd % 256 == 0
        assert both == 0 if F.bank.fmt == 4 else both >= fwd + 4 * F.T * F.f
    else:
        assert fwd == 0 and both == 0


def test_ffn_calls_reject_bad_arguments_before_any_cuda_call(lib):
    F = ffn()
    p = [(i + 2) << 36 for i in range(12)]
    F.bank.w_gate, F.bank.w_up, F.bank.w_down = p[:3]
    x, y, pre, ws, dy, dx, dwg, dwu, dwd = p[3:]
    big = 1 << 34
    fw = lambda **k: lib.moe_ffn_forward(  # noqa: E731
        ctypes.byref(k.get("F", F)), k.get("x", x), k.get("y", y), k.get("pre", None),
        k.get("ws", ws), k.get("n", big), None)
    for bad in ({"x": None}, {"y": None}, {"x": x + 8}, {"y": y + 2}, {"pre": pre + 4}, {"y": x},
                {"y": p[0] + 64}, {"pre": x}, {"ws": x}, {"y": ws}):
        assert fw(**bad) == -1, bad
    assert fw(ws=None) == -5 and fw(ws=ws + 16) == -5 and fw(n=1000) == -5
    q = ffn(fmt=4, T=4)
    assert fw(F=q, pre=pre) == -2
    bw = lambda **k: lib.moe_ffn_backward(  # noqa: E731
        ctypes.byref(k.get("F", F)), k.get("x", x), k.get("dy", dy), k.get("pre", pre),
        k.get("dx", dx), k.get("dwg", dwg), k.get("dwu", dwu), k.get("dwd", dwd),
        k.get("ws", ws), k.get("n", big), None)
    for bad in ({"x": None}, {"dy": None}, {"pre": None}, {"dx": dx + 8}, {"dwd": dwd + 2},
                {"dx": None, "dwg": None, "dwu": None, "dwd": None}, {"dx": dy}, {"dwg": dwu},
                {"dwd": p[2]}, {"dwu": pre}, {"ws": pre}):
        assert bw(**bad) == -1, bad
    assert bw(ws=None) == -5
    assert bw(n=lib.moe_ffn_workspace_size(ctypes.byref(F), 0)) == -5
    assert bw(F=q) == -2
    code = ctypes.c_int32(0)
    assert lib.moe_ffn_device_status(ctypes.byref(F), ws, big, None, ctypes.byref(code), None) == -1


def test_reference_gradients_match_autograd_and_differences():
    """The plain implementation the GPU tests compare with: its gradient formulas against
    automatic differentiation and against central differences, in 64 bits."""
    torch = pytest.importorskip("torch")
    from dense_helpers import ffn_ref
    torch.manual_seed(0)
    for act in ("silu", "gelu"):
        T, d, f = 5, 8, 16
        x, wg, wu, wd, dy = (torch.randn(*s, dtype=torch.float64)
                             for s in ((T, d), (f, d), (f, d), (d, f), (T, d)))
        ref = ffn_ref(x, wg, wu, wd, act, torch.bfloat16, dy=dy)
        leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd)]
        F = torch.nn.functional
        act_fn = F.silu if act == "silu" else (lambda t: F.gelu(t, approximate="tanh"))

        def fwd(v):
            return F.linear(act_fn(F.linear(v[0], v[1])) * F.linear(v[0], v[2]), v[3])
        y = fwd(leaves)
        torch.testing.assert_close(ref["y"][0], y.detach(), rtol=1e-12, atol=1e-12)
        names = ("dx", "dw_gate", "dw_up", "dw_down")
        for i, (n, g) in enumerate(zip(names, torch.autograd.grad(y, leaves, dy))):
            torch.testing.assert_close(ref[n][0], g, rtol=1e-11, atol=1e-11)
            v = torch.randn_like(g)
            e, base = 1e-6, [t.detach() for t in leaves]
            plus, minus = ((fwd([t + s * e * v if j == i else t for j, t in enumerate(base)]) * dy).sum()
                           for s in (1, -1))
            diff, dot = (plus - minus) / (2 * e), (g * v).sum()
            assert abs(diff - dot) <= 1e-7 * (1 + dot.abs()), n


def test_ffn_struct_layout_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "abi.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_b200.h"\n'
                   'int main(void) { printf("%zu %zu\\n", sizeof(moe_ffn), offsetof(moe_ffn, bank));'
                   ' return 0; }\n')
    exe = tmp_path / "abi"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                            check=True).stdout.split()]
    assert sizes == [ctypes.sizeof(binding.MoeFfn), binding.MoeFfn.bank.offset]


class FakeStream:
    cuda_stream, device_index = 77, -1


def calls_on_a_fake_device(monkeypatch):
    """The binding's calls with CPU tensors, a library that accepts everything and a fake CUDA
    runtime. Returns (allocations, launches, torch): the raw stream that was current at each."""
    import contextlib
    torch = pytest.importorskip("torch")
    current, allocations, launches = [0], [], []

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s.cuda_stream
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(binding, "_CURRENT", (lambda: -1, lambda index: current[0]))
    new_empty = torch.Tensor.new_empty

    def noted(self, *args, **kwargs):
        allocations.append(current[0])
        return new_empty(self, *args, **kwargs)
    monkeypatch.setattr(torch.Tensor, "new_empty", noted)

    def accept(*args):
        launches.append(args[-1])
        return 0
    return allocations, launches, accept, torch


@pytest.mark.parametrize("stream", [None, FakeStream()])
def test_results_are_allocated_for_the_stream_of_the_call(monkeypatch, stream):
    """A result from the current stream's memory, written on another stream, could be a block that
    queued work of the current stream still reads."""
    from types import SimpleNamespace
    allocations, launches, accept, torch = calls_on_a_fake_device(monkeypatch)
    bf = torch.bfloat16
    ws = torch.zeros(256, dtype=torch.uint8)
    M = SimpleNamespace(call=((2, 8), (2, 4), 8, 4, bf, bf, -1, accept))
    x = torch.zeros(2, 8, dtype=bf)
    y = binding.matvec(M, x, ws, stream=stream)
    assert y.shape == (2, 4)
    F = SimpleNamespace(call=((2, 8), (2, 2, 16), bf, -1, accept, accept), d=8, f=16)
    pre = torch.zeros(2, 2, 16)
    y = binding.ffn_forward(F, x, ws, pre=pre, stream=stream)
    grads = binding.ffn_backward(F, x, y, pre, ws, stream=stream)
    assert [tuple(g.shape) for g in grads] == [(2, 8), (16, 8), (16, 8), (8, 16)]
    want = 0 if stream is None else stream.cuda_stream
    assert allocations == [want] * 6 and launches == [want] * 3


def test_matvec_refuses_a_workspace_over_its_inputs(lib):
    """A call with K in parts writes partial sums and counters while inputs are still read."""
    m = matrix(T=32, N=1000, K=10240, ldx=10240)
    p = [(i + 2) << 36 for i in range(6)]
    m.w, m.s, m.bias, x, y, ws = p
    need = lib.moe_matvec_workspace_size(ctypes.byref(m))
    assert need > 256 + 4 * 8192                         # split
    call = lambda ws: lib.moe_matvec(ctypes.byref(m), x, y, ws, need, None)  # noqa: E731
    sizes = {m.w: 1000 * 10240 // 2, m.s: 1000 * 80 * 2, m.bias: 4000, x: 32 * 10240 * 2}
    for at, size in sizes.items():
        for off in (0, size // 2 // 256 * 256, (size - 1) // 256 * 256, -256, -(need - 256)):
            assert call(at + off) == -1, (at, off)
    m.K, m.ldx = 2560, 2560                              # not split: the status words alone
    m.T, need = 1, 256
    assert lib.moe_matvec_workspace_size(ctypes.byref(m)) == need
    assert call(x) == -1 and call(m.w) == -1


def test_matvec_takes_columns_of_one_array(lib):
    """Rows of x and y that interleave without sharing an element (slices of one wider array) are
    no overlap; one element shared is. (-3: passed on to CUDA, which has no device here.)"""
    m = matrix(T=8, N=1000, K=2560, ldx=4096, ldy=4096)
    m.w, m.s, ws, buf = ((i + 2) << 36 for i in range(4))
    size = lib.moe_matvec_workspace_size(ctypes.byref(m))
    need = max(size, 256)
    bad = lambda x, y: lib.moe_matvec(ctypes.byref(m), x, y, ws, need, None) == -1  # noqa: E731
    assert bad(buf, buf + 2 * 2559) and bad(buf, buf + 2 * 3097)  # x's end; the next row's start
    assert bad(buf + 2 * 1000, buf + 2 * 3097 + 2 * 1000 - 2 * 4096)
    assert bad(buf + 2 * 992, buf) and bad(buf, buf)
    m.y_type = 2                                                # fp32 rows twice as far apart
    assert bad(buf, buf + 2 * 2560)
    m.y_type, m.ldy = 0, 4100                                   # rows that drift into x's
    assert bad(buf, buf + 2 * 2560 + 2 * 530)
    import torch
    if not torch.cuda.is_available():
        m.ldy = 4096
        for x, y in ((buf, buf + 2 * 2560), (buf, buf + 2 * 3096), (buf + 2 * 1000, buf),
                     (buf + 2 * 1536, buf)):
            assert lib.moe_matvec(ctypes.byref(m), x, y, ws, need, None) == -3


@pytest.mark.parametrize("kind", ["matrix", "block"])
def test_a_descriptor_lets_go_of_the_weights(lib, kind):
    """Weights are freed with the last descriptor, without the garbage collector (which GPU memory
    does not wake), and live as long as one."""
    import gc
    import weakref
    torch = pytest.importorskip("torch")
    if kind == "matrix":
        owner = binding.QuantMatrix.__new__(binding.QuantMatrix)
        owner.codes, owner.bias = torch.zeros(4, 16, dtype=torch.int32), None
        owner.scales = torch.zeros(4, 1, dtype=torch.bfloat16)
        owner.N, owner.K, owner.group, owner.device = 4, 128, 128, torch.device("cpu")
    else:
        owner = binding.DeviceFfn.__new__(binding.DeviceFfn)
        w = torch.zeros(8, 8, dtype=torch.bfloat16)
        owner.bank = dict(fmt="bf16", group=128, n_exp=1, w_gate=w, w_up=w, w_down=w)
        owner.d, owner.f, owner.act, owner.dtype, owner.device = 8, 8, "silu", w.dtype, w.device
    alive, desc = weakref.ref(owner), owner.descriptor(1)
    on = gc.isenabled()
    gc.disable()
    try:
        del owner
        assert alive() is not None
        del desc
        assert alive() is None
    finally:
        if on:
            gc.enable()


def test_failure_injection_is_checked(lib):
    assert lib.moe_test_inject_dense_hold(1, -1) == -1
    assert lib.moe_test_inject_dense_hold(1, 1000) == 0
    assert lib.moe_test_inject_dense_hold(0, 0) == 0


def test_the_plain_dequantisation_is_the_oracles():
    """The weights that the GPU tests compare with, against the oracle's reading of the same words
    (every nibble value, the sign bit of a word included)."""
    import numpy as np
    torch = pytest.importorskip("torch")
    from dense_helpers import dequantise, pack
    from oracle import moe_oracle as O
    gen = torch.Generator().manual_seed(2)
    q = torch.randint(-8, 8, (24, 512), generator=gen)
    words = pack(q)
    assert (words < 0).any() and (words > 0).any() and len(q.unique()) == 16
    for group in (32, 64, 128):
        s = torch.randn(24, 512 // group, generator=gen).to(torch.bfloat16)
        W = O.dequantize(words.numpy().view(np.uint32), s.view(torch.int16).numpy().view(np.uint16),
                         "int4", group, 512)
        assert np.array_equal(W, dequantise(words, s, group).numpy())
        assert np.array_equal(W, (q.double() * s.double().repeat_interleave(group, 1)).numpy())


def test_results_are_marked_as_used_by_the_callers_stream(monkeypatch):
    """A result belongs to the given stream, but the caller reads it on another: dropped there, it
    waits for both."""
    from types import SimpleNamespace
    allocations, launches, accept, torch = calls_on_a_fake_device(monkeypatch)
    marked = []
    monkeypatch.setattr(binding, "_used_here", lambda s, *ts: marked.append(
        (binding._CURRENT[1](-1), s, [tuple(t.shape) for t in ts])))
    bf, s = torch.bfloat16, FakeStream()
    ws, x = torch.zeros(256, dtype=torch.uint8), torch.zeros(2, 8, dtype=bf)
    M = SimpleNamespace(call=((2, 8), (2, 4), 8, 4, bf, bf, -1, accept))
    F = SimpleNamespace(call=((2, 8), (2, 2, 16), bf, -1, accept, accept), d=8, f=16)
    pre = torch.zeros(2, 2, 16)
    binding.matvec(M, x, ws, stream=s)
    y = binding.ffn_forward(F, x, ws, pre=pre, stream=s)
    binding.ffn_backward(F, x, y, pre, ws, need_dw=False, stream=s)
    assert marked == [(0, s, [(2, 4)]), (0, s, [(2, 8)]), (0, s, [(2, 8)])]
