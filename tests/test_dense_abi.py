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
    dev = x.device
    binding._check_rows(x, "x", 4, 8, torch.bfloat16, dev)
    for t in (x[:, ::2], x.T, x.float(), x[:3], x[:1].expand(4, 8)):
        with pytest.raises(ValueError):
            binding._check_rows(t, "x", 4, 8, torch.bfloat16, dev)
