"""The convolution on no tokens: the state passes on, sums are zero, and only kernels that ran are counted."""
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


@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_tokens(K, given, dtype):
    N, C = 3, 20
    x, w, b = torch.zeros((N, 0, C), device="cuda", dtype=dtype), torch.randn((C, K), device="cuda"), torch.ones(C, device="cuda")
    state0, ds = (torch.randn((N, K - 1, C), device="cuda").to(dtype) for _ in range(2))
    before = ttm.launch_count()
    y, state = ttm.causal_conv_fwd(x, w, b, state0=state0 if given else None)
    assert ttm.launch_count() - before == (K > 1)
    assert y.shape == x.shape and torch.equal(state, state0 if given else torch.zeros_like(state0))
    before = ttm.launch_count()
    g = ttm.causal_conv_bwd(x, x, w, b, state0=state0 if given else None, dstate=ds)
    assert ttm.launch_count() - before == (given and K > 1)
    assert g["dx"].shape == x.shape and not g["dw"].any() and not g["db"].any()
    assert torch.equal(g["dstate0"], ds) if given else g["dstate0"] is None
    before = ttm.launch_count()
    assert ttm.causal_conv_fwd(x, w, b, want_state=False)[1] is None and ttm.launch_count() == before
