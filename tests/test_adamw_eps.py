"""AdamW with an eps next to fp32's smallest numbers: values without a gradient so far are left to the decay."""
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


@pytest.mark.parametrize("eps", [1.4e-45, 1e-40, 1e-38, 2.0 ** -126, 1.2e-38, 1e-30])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [5, 512])
def test_zero_gradients(bits, eps, n):
    """Rounding of the decay: two units of the weight, 2^-23."""
    p = torch.linspace(-2, 2, n, device="cuda")
    before = p.double()
    state = ttm.adamw_state([p], bits=bits)
    for _ in range(3):
        ttm.adamw_step([p], [torch.zeros_like(p)], state, lr=0.25, weight_decay=0.5, eps=eps)
        before = before * (1 - 0.25 * 0.5)
    assert ((p.double() - before).abs() <= 3 * 2.0 ** -23 * before.abs()).all(), p


@pytest.mark.parametrize("eps", [1e-40, 1e-38, 2.0 ** -126, 1e-20])
def test_first_steps(eps):
    """A first step is the rate in the gradient's direction wherever its square is a number of 32 bits (24 units of
    2^-24, as for any update); a gradient of zero beside it moves nothing."""
    g = torch.tensor([1.0, -1e-3, 0.0, 1e-10, -1e-15, 0.0, 1e10, 0.0], device="cuda")
    p = torch.zeros(8, device="cuda")
    ttm.adamw_step([p], [g], ttm.adamw_state([p]), lr=0.5, eps=eps)
    assert ((p + 0.5 * g.sign() * (g.abs() / (g.abs() + eps))).abs() <= 0.5 * 24 * 2.0 ** -24).all(), p
