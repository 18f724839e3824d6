"""Failure detection of the dense operators without a GPU fault: bounded waits are made to run
out, the kernels record it, wait for their copies and return, and the host reads code and site;
the same workspace, zeroed, then gives the bits it gave before."""
import pytest

torch = pytest.importorskip("torch")
from dense_helpers import quantise

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
MOE_ERR_TIMEOUT = -4
BUDGET_CYCLES = 20000  # about 10 microseconds


@pytest.fixture(scope="module")
def B():
    from expert_routed_ffn_route_b200 import binding
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load_library()
    return binding


@pytest.fixture
def hold(B):
    yield lambda on: B.test_inject_dense_hold(on, BUDGET_CYCLES)
    B.test_inject_dense_hold(False)


def run_out(B, hold, call, ws, status, site):
    """call() -> tensors, with the workspace `ws`; status() -> (code, site)."""
    want = [t.clone() for t in call()]
    assert status() == (0, 0)
    hold(True)
    call()
    torch.cuda.synchronize()
    hold(False)
    assert status() == (MOE_ERR_TIMEOUT, site)
    assert status() == (0, 0)  # read and cleared
    ws.zero_()
    for _ in range(3):
        got = call()
        assert status() == (0, 0)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,N,K,group,split", [(1, 4000, 2560, 128, False), (7, 40000, 1280, 128, False),
                                               (32, 1000, 10240, 32, True)])
def test_a_copy_of_the_matrix_never_lands(B, hold, T, N, K, group, split):
    gen = torch.Generator().manual_seed(N)
    codes, scales = quantise(gen, N, K, group)
    desc = B.QuantMatrix(codes.cuda(), scales.cuda(), K, group).descriptor(T)
    ws = B.alloc_matvec_workspace(desc)
    assert (ws.numel() > 256) == split
    x = torch.randn(T, K, generator=gen).to(BF).cuda()
    run_out(B, hold, lambda: (B.matvec(desc, x, ws),), ws,
            lambda: B.matvec_device_status(desc, ws), 60)


@pytest.mark.parametrize("T,d,f", [(8, 2560, 1024), (200, 1032, 2056), (700, 520, 1288)])
def test_a_wait_of_the_block_runs_out(B, hold, T, d, f):
    """A streamed forward pass (up to 32 rows), forward and backward on the tensor cores with and
    without tiles in parts."""
    gen = torch.Generator().manual_seed(T)
    bank = dict(fmt="bf16")
    for m, N, K in (("gate", f, d), ("up", f, d), ("down", d, f)):
        bank["w_" + m] = (torch.randn(N, K, generator=gen) * K ** -0.5).to(BF).cuda()
    desc = B.DeviceFfn(bank, d, f).descriptor(T)
    x, dy = (torch.randn(T, d, generator=gen).to(BF).cuda() for _ in range(2))
    ws = B.alloc_ffn_workspace(desc, backward=T > 32)
    pre = B.ffn_pre(desc)

    def step():
        if T <= 32:
            return (B.ffn_forward(desc, x, ws),)
        y = B.ffn_forward(desc, x, ws, pre=pre)
        return (y, *B.ffn_backward(desc, x, dy, pre, ws))
    run_out(B, hold, step, ws, lambda: B.ffn_device_status(desc, ws), 60 if T <= 32 else 51)
