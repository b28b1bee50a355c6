"""AdamW over many tensors against float64, and in 8 bits against the same arithmetic in 32 bits.

Tolerances for 32-bit moments, elementwise, u = 2^-24.  m: two products, a sum and three rounded constants or
inputs err by at most 5 u of the sum of sizes; v by 8 u of itself (a square, two products, a sum, constants); its
root by half of that and u.  1 - b^t comes from expm1 of a rounded t log b: 4 u of it.  So the update
errs by 24 u of itself and by what m's error makes of it, the weight by 4 u of itself more.  8 bits: the moments are
rounded to one of two neighbours by comparing 32-bit values, so equal arithmetic gives equal bytes."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def make(sizes, param="f32", grad="f32", packed=False, seed=0):
    r = torch.Generator().manual_seed(seed)
    p = [torch.randn(n, generator=r).to(DT[param]) for n in sizes]
    g = [(torch.randn(n, generator=r) * 10.0 ** float(torch.randint(-4, 2, (1,), generator=r))).to(DT[grad]) for n in sizes]
    if not packed:
        return [t.cuda() for t in p], [t.cuda() for t in g]
    flat = torch.cat(p).cuda()                          # neighbours in one buffer, at any address
    at = [sum(sizes[:i]) for i in range(len(sizes))]
    return [flat[a:a + n] for a, n in zip(at, sizes)], [t.cuda() for t in g]


def starts(sizes):
    at, out = 0, []
    for n in sizes:
        out.append(at)
        at += (n + 255) // 256 * 256
    return out


def plain(p, g, m, v, t, scale=1.0, lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1):
    """One step of one tensor in float64: values and tolerances."""
    b1, b2 = betas
    p, g = p.double(), g.double() * scale
    m2 = b1 * m + (1 - b1) * g
    v2 = b2 * v + (1 - b2) * g * g
    em = 5 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    den = torch.sqrt(v2 / (1 - b2 ** t)) + eps
    up = lr * m2 / (1 - b1 ** t) / den
    new = p * (1 - lr * weight_decay) - up
    return (m2, em), (v2, 8 * U * v2), (new, 24 * U * up.abs() + lr * em / (1 - b1 ** t) / den + 4 * U * p.abs())


def near(got, ref, tol, dtype=torch.float32):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol + half * (ref.abs() + tol) + 1e-37)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


SIZES = [[1], [7, 256, 255, 257], [1000, 3, 4096, 5], [2048, 2048, 2049], [100001], list(range(1, 60)),
         [0, 5, 0, 300], [33] * 700]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("param,grad,copies", [("f32", "f32", False), ("f32", "bf16", True), ("bf16", "bf16", False),
                                               ("bf16", "f32", True)])
@pytest.mark.parametrize("packed", [False, True])
def test_32_bits(sizes, param, grad, copies, packed):
    params, grads = make(sizes, param, grad, packed, seed=len(sizes))
    state = ttm.adamw_state(params)
    out = [torch.zeros_like(p, dtype=torch.bfloat16) for p in params] if copies else None
    scale = torch.tensor(0.3, device="cuda")
    for t in (1, 2, 3):
        # each step from what the one before left
        before = [p.clone() for p in params]
        m0, v0 = state["m"].clone(), state["v"].clone()
        ttm.adamw_step(params, grads, state, grad_scale=scale, copies=out, **HYPER)
        for i, (a, n) in enumerate(zip(starts(sizes), sizes)):
            m, v, p = plain(before[i].cpu(), grads[i].cpu(), m0[a:a + n].double().cpu(), v0[a:a + n].double().cpu(), t,
                            float(scale))
            near(state["m"][a:a + n], *m)
            near(state["v"][a:a + n], *v)
            near(params[i], *p, DT[param])
            if copies:
                near(out[i], *p, torch.bfloat16)
            assert not state["m"][a + n:a + (n + 255) // 256 * 256].any()
    assert state["step"].tolist() == [3, 0]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_moments_round_after_every_operation(grad):
    """m and v in 32 bits are those of single operations, bit for bit: none is fused with the next."""
    p, g = make([5000, 257, 70001], "f32", grad, seed=6)
    state = ttm.adamw_state(p)
    b1, b2 = torch.tensor(0.9, device="cuda"), torch.tensor(0.95, device="cuda")
    c1, c2 = torch.tensor(1 - 0.9, device="cuda"), torch.tensor(1 - 0.95, device="cuda")
    want = [(torch.zeros_like(a), torch.zeros_like(a)) for a in p]
    for _ in range(3):
        ttm.adamw_step(p, g, state, **HYPER)
        want = [(m * b1 + x.float() * c1, v * b2 + (x.float() * x.float()) * c2) for (m, v), x in zip(want, g)]
    for (m, v), at in zip(want, starts([5000, 257, 70001])):
        assert torch.equal(state["m"].flatten()[at:at + m.numel()], m)
        assert torch.equal(state["v"].flatten()[at:at + v.numel()], v)


def dither(first, n, t):
    at = first + torch.arange(n)
    h = (at + t * 0x9e3779b9) & 0xffffffff
    h ^= h >> 16
    h = h * 0x7feb352d & 0xffffffff
    h ^= h >> 15
    h = h * 0x846ca68b & 0xffffffff
    h ^= h >> 16
    return (h & 0xffff).float() / 65536, (h >> 16).float() / 65536


def to_8(x, frac):
    """Blocks of 256 in e4m3, element by element by frexp: codes as values, and the scales."""
    n = x.numel()
    x = torch.cat((x, torch.zeros(-n % 256))).view(-1, 256)
    frac = torch.cat((frac, torch.zeros(-n % 256))).view(-1, 256)
    most = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(1)
    f, e = torch.frexp(most)                            # most = f 2^e, f in [0.5, 1)
    e = torch.where(most > 0, e - 9 + (f > 0.875).int(), torch.tensor(-126)).clamp(min=-126)
    y = torch.ldexp(x.abs(), -e[:, None])
    _, b = torch.frexp(y)
    step = torch.where(y > 0, b - 4, torch.tensor(-9)).clamp(min=-9)
    q = torch.ldexp(torch.floor(torch.ldexp(y, -step) + frac), step)
    q = torch.where(torch.isfinite(x), torch.copysign(q, x), float("nan"))
    return q.view(-1)[:n], torch.ldexp(torch.ones(()), e)


@pytest.mark.parametrize("sizes", [[1], [256], [7, 300, 2048, 5000], [65536]])
@pytest.mark.parametrize("grad,packed", [("f32", False), ("bf16", True)])
def test_8_bits(sizes, grad, packed):
    params, grads = make(sizes, "f32", grad, packed, seed=9)
    state = ttm.adamw_state(params, bits=8)
    b1, b2 = (torch.tensor(b, dtype=torch.float32) for b in HYPER["betas"])
    c1, c2 = (torch.tensor(1 - b, dtype=torch.float32) for b in HYPER["betas"])
    mv = [(torch.zeros(n), torch.zeros(n)) for n in sizes]
    for t in range(1, 6):
        before = [p.cpu() for p in params]
        # gradients of growing and shrinking size
        grads = [g * s for g, s in zip(grads, [1.0 if t < 3 else 0.01] * len(grads))]
        ttm.adamw_step(params, grads, state, **HYPER)
        m_out, v_out = ttm.adamw_moments(state)
        for i, (a, n) in enumerate(zip(starts(sizes), sizes)):
            g, (m, r) = grads[i].float().cpu(), mv[i]
            v = r * r
            want = plain(before[i], g, m.double(), v.double(), t)
            m = m * b1 + g * c1
            v = v * b2 + g * g * c2
            fm, fr = dither(a, n, t)
            (qm, sm), (qr, sr) = to_8(m, fm), to_8(torch.sqrt(v), fr)
            blocks = slice(a // 256, a // 256 + (n + 255) // 256)
            assert torch.equal(state["m_scale"][blocks].cpu(), sm) and torch.equal(state["v_scale"][blocks].cpu(), sr)
            assert torch.equal(state["m"][a:a + n].float().cpu(), qm)
            assert torch.equal(state["v"][a:a + n].float().cpu(), qr)
            mv[i] = ((qm.view(-1) * sm.repeat_interleave(256)[:n]), qr * sr.repeat_interleave(256)[:n])
            assert torch.equal(m_out[a:a + n].cpu(), mv[i][0]) and torch.equal(v_out[a:a + n].cpu(), mv[i][1] ** 2)
            near(params[i], *want[2])
            # a value moves by less than a step of its binade, at least 2^-9 of the scale
            step = torch.maximum(want[0][0].abs() / 8, sm.repeat_interleave(256)[:n].double() / 512)
            assert ((mv[i][0].double() - want[0][0]).abs() <= step * (1 + 1e-6)).all()


def test_8_bit_moments_do_not_stand_still():
    """A constant gradient: m approaches it by a tenth a step on average over 65536 values.  A rounding errs by
    less than a step, 1/8 of the value, and evenly; of the errors a share of 0.9 a step stays: the mean's spread is
    at most (1/8) / sqrt(1 - 0.81) / sqrt(65536) = 1.1e-3 of the gradient, and 6 times that is the bound."""
    n = 65536
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    state = ttm.adamw_state([p], bits=8)
    for t in range(1, 60):
        ttm.adamw_step([p], [g], state, lr=0.0, weight_decay=0.0)
        m, v = ttm.adamw_moments(state)
        if t in (1, 5, 20, 59):
            assert abs(float(m.mean()) - (1 - 0.9 ** t)) < 6.6e-3, t
    assert not p.any()                                  # lr 0


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_that_are_missing_or_not_finite(bits):
    params, grads = make([300, 40, 600], seed=2)
    state = ttm.adamw_state(params, bits=bits)
    ttm.adamw_step(params, grads, state, **HYPER)
    keep = params[1].clone(), state["m"].clone(), state["v"].clone()
    ttm.adamw_step(params, [grads[0], None, grads[2]], state, **HYPER)
    assert torch.equal(params[1], keep[0])
    for a, b in ((state["m"], keep[1]), (state["v"], keep[2])):
        a, b = a.view(torch.uint8), b.view(torch.uint8)
        s = a.numel() // state["m"].numel()
        assert torch.equal(a[512 * s:768 * s], b[512 * s:768 * s]) and not torch.equal(a[:512 * s], b[:512 * s])
    bad = grads[0].clone()
    bad[7], bad[300 - 1] = float("nan"), float("inf")
    ttm.adamw_step(params, [bad, None, None], state, **HYPER)
    m, _ = ttm.adamw_moments(state)
    assert torch.isnan(m[7]) and not torch.isfinite(m[299]) and int((~torch.isfinite(m)).sum()) == 2
    assert int((~torch.isfinite(params[0])).sum()) == 2
    assert state["step"].tolist() == [3, 0]
    ttm.adamw_step([], [], ttm.adamw_state([torch.zeros(0, device="cuda")]) | dict(step=state["step"]), lr=1.0)
    assert state["step"].tolist() == [4, 0]


def test_zero_gradients_and_zero_moments():
    for bits in (8, 32):
        p = torch.ones(500, device="cuda")
        state = ttm.adamw_state([p], bits=bits)
        ttm.adamw_step([p], [torch.zeros_like(p)], state, lr=0.5, weight_decay=0.1)
        assert float((p - 0.95).abs().max()) < 1e-7 and not any(t.any() for t in ttm.adamw_moments(state))


def test_captured_calls_count_their_replays():
    def run(replays):
        params, grads = make([1000, 77], seed=4)
        state, lr = ttm.adamw_state(params, bits=8), torch.tensor(1e-2, device="cuda")
        if not replays:
            for i in range(6):
                ttm.adamw_step(params, grads, state, lr=1e-2 if i < 3 else 1e-3)
            return params, state
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ttm.adamw_step(params, grads, state, lr=lr)
        for i in range(6):
            if i == 3:
                lr.fill_(1e-3)
            graph.replay()
        torch.cuda.synchronize()
        return params, state
    (p, s), (q, z) = run(False), run(True)
    assert all(torch.equal(a, b) for a, b in zip(p, q)) and torch.equal(s["step"], z["step"])
    assert torch.equal(s["m"].view(torch.uint8), z["m"].view(torch.uint8))


def test_autograd_sees_the_parameters_change():
    w = torch.ones(4, device="cuda", requires_grad=True)
    loss = (w * w).sum()
    with torch.no_grad():
        ttm.adamw_step([w], [torch.ones_like(w)], ttm.adamw_state([w]), lr=0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_other_streams_and_long_runs():
    params, grads = make([5000], seed=6)
    twin, state, other = params[0].clone(), ttm.adamw_state(params), ttm.adamw_state(params)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ttm.adamw_step(params, grads, state, stream=side, **HYPER)
    side.synchronize()
    ttm.adamw_step([twin], grads, other, **HYPER)
    assert torch.equal(twin, params[0])
    # late steps: 1 - b^t is one
    other["step"][0] = 2 ** 24
    before, m0, v0 = twin.clone(), other["m"].clone(), other["v"].clone()
    ttm.adamw_step([twin], grads, other, **HYPER)
    _, _, p = plain(before.cpu(), grads[0].cpu(), m0[:5000].double().cpu(), v0[:5000].double().cpu(), 2 ** 24 + 1)
    near(twin, *p)


def test_offsets_past_32_bits():
    """A tensor of 2.2e9 values beside a short one: its last values as a tensor of their own gives them."""
    n = 2 ** 31 + 70001
    p, g = torch.ones(n, device="cuda", dtype=torch.bfloat16), torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    g[-1000:] = torch.linspace(-1, 1, 1000, device="cuda").to(torch.bfloat16)
    short, gs = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    state = ttm.adamw_state([p, short])
    end, ge = torch.ones(1000, device="cuda", dtype=torch.bfloat16), g[-1000:].clone()
    other = ttm.adamw_state([end])
    for _ in range(2):
        ttm.adamw_step([p, short], [g, gs], state, **HYPER)
        ttm.adamw_step([end], [ge], other, **HYPER)
    assert torch.equal(p[-1000:], end) and torch.equal(state["m"][n - 1000:n], other["m"][:1000])
    assert torch.equal(state["v"][n - 1000:n], other["v"][:1000]) and not state["m"][n:(n + 255) // 256 * 256].any()
    assert bool((short < 1).all()) and bool((state["m"][-512:-212] > 0).all())


def test_refusals():
    p, g = [torch.zeros(300, device="cuda")], [torch.ones(300, device="cuda")]
    state = ttm.adamw_state(p)
    flat = torch.zeros(600, device="cuda")
    pair = ttm.adamw_state([flat[:300], flat[300:]])
    two = [g[0], g[0]]
    step = lambda params=p, grads=g, s=state, **k: ttm.adamw_step(params, grads, s, **({"lr": 0.1} | k))  # noqa: E731
    bad = [lambda: ttm.adamw_state(p, bits=16), lambda: ttm.adamw_state([]), lambda: step(grads=[]), lambda: step(params=None),
           lambda: step(grads=[g[0][:299]]), lambda: step(params=[p[0][:200]], grads=[g[0][:200]]), lambda: step(params=[p[0].cpu()]),
           lambda: step(grads=[g[0].cpu()]), lambda: step(s={}), lambda: step(betas=(1.0, 0.9)), lambda: step(betas=(0.9, -0.1)),
           lambda: step(eps=0.0), lambda: step(lr=float("nan")), lambda: step(weight_decay=float("inf")),
           lambda: step(grad_scale=torch.ones(2, device="cuda")), lambda: step(grad_scale=torch.ones(())),
           lambda: step(copies=[torch.zeros(300, device="cuda")]), lambda: step(copies=[]),
           lambda: step(grads=[p[0]]),                                          # the parameter as its own gradient
           lambda: step([flat[:300], flat[:300]], two, pair), lambda: step([flat[:300], flat[299:599]], two, pair),
           lambda: step([flat[:300], flat[300:]], two, pair | dict(v=pair["m"])),
           lambda: step(s=state | dict(m=state["m"][:256])),
           lambda: step([torch.zeros(600, device="cuda")[::2]])]
    for call in bad:
        with pytest.raises(ttm.TTMError):
            call()
    for call in (lambda: step(params=[p[0].half()]), lambda: step(grads=[g[0].half()])):
        with pytest.raises((TypeError, ttm.TTMError)):
            call()
    assert not p[0].any() and state["step"].tolist() == [0, 0]
    step([flat[:300], flat[300:]], two, pair)                                   # one gradient for two parameters
    assert flat.all()
