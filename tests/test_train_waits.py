"""A device wait of the operators around the scan that runs out: the call ends, the status word says so
once, and the next call is right again.  The wait is made to run out by a product that is not announced or a
copy that is announced 16 bytes too long; nothing faults or hangs."""
import time

import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def stalls(call, at):
    """The clean result of the call, then one with its wait `at` running out, then a clean one again."""
    want = call()
    assert ttm.device_status() == ttm.OK
    ttm.debug_set("wait_cycles", 20_000_000)          # ~10 ms at 2 GHz
    ttm.debug_set("stall_chunk", at)
    try:
        t0 = time.perf_counter()
        call()
        status = ttm.device_status()                  # synchronises
        assert status == ttm.ERR_TIMEOUT, ttm.status_str(status)
        assert time.perf_counter() - t0 < 10.0
        assert ttm.device_status() == ttm.OK          # the query cleared it
    finally:
        ttm.debug_set("stall_chunk", -1)
        ttm.debug_set("wait_cycles", 0)
    got = call()
    assert ttm.device_status() == ttm.OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("batch,m,n,at", [(3, 64, 64, 0), (400, 100, 128, 4), (3, 128, 40, 14),     # a block a matrix
                                          (2, 60, 700, 0), (2, 60, 700, 1), (3, 1000, 64, 5),       # a cluster
                                          (2, 33, 260, 14), (1, 5, 200, 13),
                                          (2, 100, 900, 0), (2, 100, 900, 4), (1, 3000, 50, 2),     # A alone
                                          (1, 300, 500, 0), (2, 500, 300, 5), (1, 1100, 1300, 3)])  # products
def test_orthogonalize(batch, m, n, at):
    G = torch.randn((batch, m, n), generator=torch.Generator().manual_seed(m)).cuda()
    stalls(lambda: (ttm.orthogonalize(G),), at)


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("N,T,D,dtype,at", [(2, 777, 768, "bf16", 3), (2, 5000, 128, "bf16", 0), (1, 40000, 64, "f32", 7),
                                            (3, 1500, 40, "bf16", 2), (30, 9000, 64, "bf16", 40)])
def test_recurrence(N, T, D, dtype, at, token):
    """One of the tiles never arrives: its block leaves, and the blocks that wait for its state give up too."""
    r = torch.Generator().manual_seed(T)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = torch.randn((N, T, D), generator=r).to(dt).cuda()
    g = (-0.1 * torch.rand((N, T) if token else (N, T, D), generator=r)).to(torch.float32 if token else dt).cuda()
    h, _ = ttm.glr_fwd(x, g)
    stalls(lambda: ttm.glr_fwd(x, g), at)
    stalls(lambda: tuple(ttm.glr_bwd(g, h, x).values()), at)
