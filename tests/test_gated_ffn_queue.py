"""The feed-forward block behind work that is still running, and on a single row however far the next would be."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def make(N, D, F):
    r = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(s, generator=r, device="cuda").to(BF)  # noqa: E731
    return rand(N, D), rand(N, D), rand(D, 2 * F) / D ** 0.5, rand(F, D) / F ** 0.5


@pytest.mark.parametrize("N,D,F", [(1, 64, 96), (16, 256, 512), (128, 512, 640), (300, 256, 512), (1100, 256, 512)])
def test_a_wait_counts_from_the_end_of_the_work_before(N, D, F):
    """An optimiser step of 1.5 ms (10 GB) lets the next kernel start beside it; the limit of a wait is 0.5 ms at 2 GHz."""
    x, dy, W_in, W_out = make(N, D, F)
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)
    n = 400_000_000
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda", dtype=BF)
    state = ttm.adamw_state([p])
    ttm.adamw_step([p], [g], state, lr=1e-3)
    assert ttm.device_status() == ttm.OK
    ttm.debug_set("wait_cycles", 1_000_000)
    try:
        for _ in range(3):
            ttm.adamw_step([p], [g], state, lr=1e-3)
            y2, gu2 = ttm.gated_ffn_fwd(x, W_in, W_out)
            ttm.adamw_step([p], [g], state, lr=1e-3)
            d2 = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)
        status = ttm.device_status()                  # synchronises
    finally:
        ttm.debug_set("wait_cycles", 0)
    assert status == ttm.OK, ttm.status_str(status)
    assert torch.equal(y2, y) and torch.equal(gu2, gu) and all(torch.equal(d[k], d2[k]) for k in d)


@pytest.mark.parametrize("row", [0, 8, 64, 1 << 20, 1 << 42])
def test_one_row_has_no_next(row):
    """The distance between rows says nothing where there is one."""
    L, (N, D, F) = ttm.lib(), (1, 64, 96)
    x, dy, W_in, W_out = make(N, D, F)
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out, residual=dy)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)
    out = [torch.zeros_like(t) for t in (y, gu, *d.values())]
    n = max(L.ttm_gated_ffn_workspace_size(N, D, F, b) for b in (0, 1))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    at = [t.data_ptr() for t in (x, dy, W_in, W_out, *out, ws)]
    assert L.ttm_gated_ffn_fwd(N, D, F, 0, at[0], row, at[2], at[3], at[1], row, at[4], at[5], at[9], n, s) == ttm.OK
    assert L.ttm_gated_ffn_bwd(N, D, F, 0, at[1], row, at[0], row, at[5], at[2], at[3], at[6], at[7], at[8], at[9], n,
                               s) == ttm.OK
    assert all(torch.equal(a, b) for a, b in zip(out, (y, gu, *d.values())))
