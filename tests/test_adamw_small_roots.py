"""AdamW with moments in 8 bits where one block of 256 values holds gradients of very different sizes: the codes and
scales against the same arithmetic in 32 bits, and the size of the steps."""
import pytest
import torch

import test_neural_memory_gb300 as ttm
from tests.test_adamw import HYPER, near, plain, starts, to_8

pytestmark = pytest.mark.gpu
LOWEST = 2.0 ** -9                    # e4m3's smallest size


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def dither(first, n, t):
    """The hash's two halves for the places first .. first + n - 1 of the moments, as fractions."""
    at = first + torch.arange(n)
    h = (at + t * 0x9e3779b9 + (at >> 32) * 0x85ebca6b) & 0xffffffff
    h ^= h >> 16
    h = h * 0x7feb352d & 0xffffffff
    h ^= h >> 15
    h = h * 0x846ca68b & 0xffffffff
    h ^= h >> 16
    return (h & 0xffff).float() / 65536, (h >> 16).float() / 65536


def coded(m, v, first, t):
    """Codes and scales of m and sqrt(v); a root is not coded as zero beside an m that is not."""
    n, root = m.numel(), torch.sqrt(v)
    fm, fr = dither(first, n, t)
    (qm, sm), (qr, sr) = to_8(m, fm), to_8(root, fr)
    return (qm, sm), (torch.where((qr == 0) & (qm != 0), LOWEST, qr), sr)


def spread(sigma, zeros=0.0):
    """Gradients of sizes exp(sigma * normal), a share of them zero at every step."""
    def make(n, r):
        size = 1e-3 * torch.exp(sigma * torch.randn(n, generator=r))
        return lambda: size * torch.randn(n, generator=r) * (torch.rand(n, generator=r) >= zeros)
    return make


def one_large(small, zeros=0.0):
    """A gradient of size 1 in every block, the others `small`."""
    def make(n, r):
        size = torch.full((n,), small)
        size[::256] = 1.0
        return lambda: size * torch.randn(n, generator=r) * (torch.rand(n, generator=r) >= zeros)
    return make


KINDS = {"exp1": spread(1.0), "exp2": spread(2.0), "exp3": spread(3.0), "exp5": spread(5.0), "exp3 zeros": spread(3.0, 0.5),
         "3e-5 zeros": one_large(3e-5, 0.5), "1e-5": one_large(1e-5)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,packed", [([7, 300, 4096, 5000], False), ([7, 300, 4096, 5000], True)])
def test_codes_of_blocks_of_many_sizes(kind, sizes, packed):
    r = torch.Generator().manual_seed(3)
    draws = [KINDS[kind](n, r) for n in sizes]
    flat = torch.randn(sum(sizes), generator=r).cuda()
    at = [sum(sizes[:i]) for i in range(len(sizes))]
    params = [flat[a:a + n] if packed else flat[a:a + n].clone() for a, n in zip(at, sizes)]
    state = ttm.adamw_state(params, bits=8)
    b1, b2 = (torch.tensor(b, dtype=torch.float32) for b in HYPER["betas"])
    c1, c2 = (torch.tensor(1 - b, dtype=torch.float32) for b in HYPER["betas"])
    mv = [(torch.zeros(n), torch.zeros(n)) for n in sizes]
    raised = 0
    for t in range(1, 13):
        before, grads = [p.cpu() for p in params], [d() for d in draws]
        ttm.adamw_step(params, [g.cuda() for g in grads], state, **HYPER)
        m_out, v_out = ttm.adamw_moments(state)
        for i, (a, n) in enumerate(zip(starts(sizes), sizes)):
            g, (m, q) = grads[i], mv[i]
            want = plain(before[i], g, m.double(), (q * q).double(), t)
            m, v = m * b1 + g * c1, (q * q) * b2 + g * g * c2
            (qm, sm), (qr, sr) = coded(m, v, a, t)
            raised += int(((qr == LOWEST) & (qm != 0)).sum())
            blocks = slice(a // 256, a // 256 + (n + 255) // 256)
            assert torch.equal(state["m_scale"][blocks].cpu(), sm) and torch.equal(state["v_scale"][blocks].cpu(), sr)
            assert torch.equal(state["m"][a:a + n].float().cpu(), qm)
            assert torch.equal(state["v"][a:a + n].float().cpu(), qr)
            mv[i] = qm * sm.repeat_interleave(256)[:n], qr * sr.repeat_interleave(256)[:n]
            assert torch.equal(m_out[a:a + n].cpu(), mv[i][0]) and torch.equal(v_out[a:a + n].cpu(), mv[i][1] ** 2)
            near(params[i], *want[2])
    assert raised or kind == "exp1"


@pytest.mark.parametrize("kind", KINDS)
def test_steps_stay_near_the_learning_rate(kind):
    """In 32 bits |m| / sqrt(v) is at most c1 / sqrt(c2 (1 - b1^2 / b2)) = 1.2 with the bias corrections settled.  In 8 bits a
    root may be one code too low while m is one too high: at worst 2 steps of e4m3's smallest size go to 1 and |m| to 1.2 * 2 + 1,
    a ratio of 3.4 (a scale of m twice that of the root: 4.4), and errors of earlier steps add to it while they decay.  Eight
    times the rate is the bound; a root coded as zero under an m that is not takes hundreds."""
    n = 64 * 256
    r = torch.Generator().manual_seed(11)
    draw = KINDS[kind](n, r)
    p = torch.zeros(n, device="cuda")
    state = ttm.adamw_state([p], bits=8)
    worst = torch.zeros((), device="cuda")
    for _ in range(250):
        before = p.clone()
        ttm.adamw_step([p], [draw().cuda()], state, lr=1.0, weight_decay=0.0)
        worst = torch.maximum(worst, (p - before).abs().max())
    assert float(worst) < 8.0, float(worst)


def test_places_past_32_bits():
    """The dither of values behind 2^32 others, whose tensor has no gradient and stays as it is."""
    n, m = 2 ** 32 + 512, 5000
    big = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    r = torch.Generator().manual_seed(5)
    p, g = torch.randn(m, generator=r), torch.randn(m, generator=r)
    small, state = p.cuda(), ttm.adamw_state([big, p.cuda()], bits=8)
    b1, b2 = (torch.tensor(b, dtype=torch.float32) for b in HYPER["betas"])
    c1, c2 = (torch.tensor(1 - b, dtype=torch.float32) for b in HYPER["betas"])
    mq = vq = torch.zeros(m)
    for t in (1, 2, 3):
        ttm.adamw_step([big, small], [None, g.cuda()], state, **HYPER)
        (qm, sm), (qr, sr) = coded(mq * b1 + g * c1, vq * vq * b2 + g * g * c2, n, t)
        assert torch.equal(state["m"][n:n + m].float().cpu(), qm) and torch.equal(state["v"][n:n + m].float().cpu(), qr)
        assert torch.equal(state["m_scale"][n // 256:].cpu(), sm) and torch.equal(state["v_scale"][n // 256:].cpu(), sr)
        mq, vq = qm * sm.repeat_interleave(256)[:m], qr * sr.repeat_interleave(256)[:m]
    assert not state["m"][:n].view(torch.int64).any() and not big.view(torch.int64).any()
