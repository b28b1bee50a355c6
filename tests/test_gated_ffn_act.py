"""The activations of the gated feed-forward block on every bf16 value, against float64.

With u = 1 and an output product that is the identity the result is act(g) rounded to bf16: half a step, 2^-8 of itself,
on top of fp32 errors.  SiLU: (4 + 0.7 |g|) 2^-23 of the logistic, a product.  GELU: the tail's polynomial is 2e-6 of itself
off, less than 2^-18; its exponent g^2 / 2, of two roundings in base 2, errs by (g^2 / 2) 2^-22 of the result, the exponential
and the reciprocal by 2^-22 each (the polynomial's own slope carries less on).  What is below the smallest normal number
may be taken as zero."""
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


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [40, 4096])            # through the kernel of few rows and of many
def test_every_bf16_value(act, rows):
    g = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    g = g[torch.isfinite(g)].cuda()
    g = torch.where(g.abs() < 1e30, g, torch.ones_like(g))
    D = 64
    # columns 0 .. 62 of x hold gates, column 63 a one that makes every u
    n = (g.numel() + 62) // 63
    x = torch.ones((n, D), device="cuda", dtype=BF)
    x[:, :63] = torch.cat((g, g[:n * 63 - g.numel()])).view(n, 63)
    W_in = torch.zeros((D, 2 * D), device="cuda", dtype=BF)
    W_in[:63, :63] = torch.eye(63)
    W_in[63, D:] = 1
    y = torch.cat([ttm.gated_ffn_fwd(x[a:a + rows].contiguous(), W_in, torch.eye(D, device="cuda", dtype=BF), act=act)[0]
                   for a in range(0, n, rows)])
    got, v = y[:, :63].reshape(-1)[:g.numel()].double(), g.double()
    if act == "silu":
        want, rel = v * torch.sigmoid(v), (6 + 0.7 * v.abs().clamp_max(200)) * 2.0 ** -23
    else:
        want = v * 0.5 * torch.erfc(-v / 2 ** 0.5)
        rel = 2.0 ** -18 + (0.5 * v * v).clamp_max(200) * 2.0 ** -22 + 2.0 ** -20
    bad = ~((got - want).abs() <= want.abs() * (2.0 ** -8 + 1.01 * rel) + 2.0 ** -126 * (1 + v.abs()))
    assert not bad.any(), (int(bad.sum()), v[bad][:8].tolist(), got[bad][:8].tolist(), want[bad][:8].tolist())
