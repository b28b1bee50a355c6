"""Gated linear recurrence (glr_fwd, glr_bwd, glr_step) against a float64 token loop.

Tolerances, elementwise.  A retention over j tokens is a product of j values of exp, each
good to 2 units in the last place, so a term x_s reaches h_t with a relative error of at
most (t - s + 4) 2^-22; with m_t = a m_{t-1} + |x_t| and p_t = a (p_{t-1} + m_{t-1}) (that
is, sum over s of (t - s) times its term) the fp32 value is off by at most 2^-22 (p_t + 4 m_t),
taken twice for the sums' own rounding.  A bf16 output (8 significant bits) adds half a unit, 2^-8 of its value."""
import math

import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
U = 2.0 ** -21
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def make(N, T, D, dtype, token, seed=0, resets=False, h0=True, keep_all=False):
    r = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    x = torch.randn((N, T, D), generator=r).to(dt)
    shape = (N, T) if token else (N, T, D)
    alpha = 0.3 * torch.rand(shape, generator=r)
    g = torch.zeros(shape) if keep_all else torch.log1p(-alpha)
    if resets and T:
        g.masked_fill_(torch.rand(shape, generator=r) < 0.1, -math.inf)
    g = g.to(torch.float32 if token else dt)
    s = torch.randn((N, D), generator=r) if h0 else None
    return x, g, s


def decay(g, D):
    a = torch.exp(g.double())
    return a if a.dim() == 3 else a[..., None].expand(-1, -1, D)


def reference(x, g, h0):
    """h, its tolerance's fp32 part, and both for the last token."""
    N, T, D = x.shape
    a, x = decay(g, D), x.double()
    h = torch.zeros(N, D, dtype=torch.float64) if h0 is None else h0.double()
    m, p = h.abs(), torch.zeros_like(h)
    hs, ts = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        p = a[:, t] * (p + m)
        m = a[:, t] * m + x[:, t].abs()
        h = a[:, t] * h + x[:, t]
        hs[:, t], ts[:, t] = h, U * (p + 4 * m)
    return hs, ts, h, U * (p + 4 * m)


def close(got, ref, tol, dtype):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    bad = (got - ref).abs() > tol + HALF[dtype] * (ref.abs() + tol) + 1e-37
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


def on(t):
    return None if t is None else t.cuda()


SHAPES = [(1, 1, 1), (1, 2, 8), (2, 3, 5), (1, 17, 64), (3, 64, 128), (2, 127, 64), (2, 129, 40),
          (1, 1000, 199), (5, 513, 24), (2, 300, 136), (1, 2049, 128), (300, 9, 16), (3, 5, 2048),
          (1, 4097, 8), (1300, 20, 512), (5, 11, 131)]


@pytest.mark.parametrize("N,T,D", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("token", [False, True])
def test_forward(N, T, D, dtype, token):
    x, g, h0 = make(N, T, D, dtype, token, seed=T + D, resets=T % 2 == 1, h0=D % 3 != 1)
    h, last = ttm.glr_fwd(on(x), on(g), h0=on(h0))
    rh, th, rl, tl = reference(x, g, h0)
    close(h, rh, th, x.dtype)
    close(last, rl, tl, torch.float32)


def grad_reference(g, h, h0, dh, dh_last):
    N, T, D = dh.shape
    a, dh, h = decay(g, D), dh.double(), h.double()
    c = torch.zeros(N, D, dtype=torch.float64) if dh_last is None else dh_last.double()
    m, p = c.abs(), torch.zeros_like(c)
    zero = torch.zeros(N, D, dtype=torch.float64) if h0 is None else h0.double()
    dx, tx = torch.empty_like(dh), torch.empty_like(dh)
    dg, tg = torch.empty_like(dh), torch.empty_like(dh)
    for t in range(T - 1, -1, -1):
        G, m = dh[:, t] + c, dh[:, t].abs() + m
        dx[:, t], tx[:, t] = G, U * (p + 4 * m)
        p, m, c = a[:, t] * (p + m), a[:, t] * m, a[:, t] * G
        before = h[:, t - 1] if t else zero
        dg[:, t], tg[:, t] = c * before, U * (p + 6 * m) * before.abs()
    if g.dim() == 2:   # a sum over the channels: D more roundings at most, of the sum of sizes
        tg = (tg + D * 2.0 ** -24 * dg.abs()).sum(-1)
        dg = dg.sum(-1)
    return dx, tx, dg, tg, c, U * (p + 6 * m)


@pytest.mark.parametrize("N,T,D", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("token", [False, True])
def test_gradient(N, T, D, dtype, token):
    x, g, h0 = make(N, T, D, dtype, token, seed=T + D, resets=T % 2 == 0, h0=D % 3 != 1)
    h = reference(x, g, h0)[0].to(x.dtype)
    r = torch.Generator().manual_seed(7)
    dh = torch.randn((N, T, D), generator=r).to(x.dtype)
    last = torch.randn((N, D), generator=r) if T % 3 else None
    out = ttm.glr_bwd(on(g), on(h), on(dh), h0=on(h0), dh_last=on(last))
    dx, tx, dg, tg, c, tc = grad_reference(g, h, h0, dh, last)
    close(out["dx"], dx, tx, x.dtype)
    close(out["dg"], dg, tg, g.dtype)
    close(out["dh0"], c, tc, torch.float32)
    again = ttm.glr_bwd(on(g), on(h), on(dh), h0=on(h0), dh_last=on(last))
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("N,n,D", [(1, 1, 1), (4, 1, 64), (1000, 1, 128), (3, 2, 199), (2, 7, 2048),
                                   (65, 3, 40)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("token", [False, True])
def test_step(N, n, D, dtype, token):
    x, g, s = make(N, n, D, dtype, token, seed=N)
    state = s.cuda()
    h = ttm.glr_step(on(x), on(g), state)
    rh, th, rl, tl = reference(x, g, s)
    close(h, rh, th, x.dtype)
    close(state, rl, tl, torch.float32)


@pytest.mark.parametrize("token", [False, True])
def test_forward_in_parts_and_step_continue_it(token):
    x, g, h0 = make(2, 700, 72, "f32", token, seed=3)
    rh, th, rl, tl = reference(x, g, h0)
    h1, s = ttm.glr_fwd(on(x[:, :450]), on(g[:, :450]), h0=on(h0))
    h2, s = ttm.glr_fwd(on(x[:, 450:690]), on(g[:, 450:690]), h0=s)
    h3 = ttm.glr_step(on(x[:, 690:]), on(g[:, 690:]), s)
    # a cut rounds the state once more, which the factor of two over the sums' own bound covers
    close(torch.cat((h1, h2, h3), 1), rh, 2 * th, torch.float32)
    close(s, rl, 2 * tl, torch.float32)


@pytest.mark.parametrize("T", [300, 70001])
def test_nothing_forgotten(T):
    """g = 0: a running sum, the longest memory there is."""
    x, g, h0 = make(2, T, 24, "f32", False, keep_all=True)
    h, last = ttm.glr_fwd(on(x), on(g), h0=on(h0))
    ref = h0.double()[:, None] + x.double().cumsum(1)
    size = h0.double().abs()[:, None] + x.double().abs().cumsum(1)
    # no exp errs here (exp(0) = 1): only the order of the sum, at most 2^-24 a token
    tol = 2.0 ** -24 * (torch.arange(T)[None, :, None] + 4) * size
    close(h, ref, tol, torch.float32)
    close(last, ref[:, -1], tol[:, -1], torch.float32)


@pytest.mark.parametrize("pad,lead", [(0, 1), (8, 1), (3, 1), (8, 2), (5, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_column_slices(pad, lead, dtype):
    """x, g and dh as columns of wider rows, at aligned and odd offsets, with two leading
    dimensions; the same values as from contiguous tensors, bit for bit."""
    D, T = 48, 200
    B = (3,) if lead == 1 else (2, 3)
    r = torch.Generator().manual_seed(1)
    buf = torch.randn((*B, T, 3 * D + pad), generator=r).to(DT[dtype]).cuda()
    x, g, dh = (buf[..., i * D + min(pad, 3):(i + 1) * D + min(pad, 3)] for i in range(3))
    g.copy_(-g.float().abs() * 0.2)
    h, last = ttm.glr_fwd(x, g)
    h2, last2 = ttm.glr_fwd(x.contiguous(), g.contiguous())
    flat = lambda t: t.reshape(-1, *t.shape[-2:]).cpu()  # noqa: E731
    rh, th, rl, tl = reference(flat(x), flat(g), None)
    close(flat(h), rh, th, x.dtype)
    close(last.reshape(-1, D), rl, tl, torch.float32)
    close(flat(h2), rh, th, x.dtype)
    out = ttm.glr_bwd(g, h, dh)
    dx, tx, dg, tg, c, tc = grad_reference(flat(g), flat(h), None, flat(dh), None)
    close(flat(out["dx"]), dx, tx, x.dtype)
    close(flat(out["dg"]), dg, tg, x.dtype)
    close(out["dh0"].reshape(-1, D), c, tc, torch.float32)
    state = torch.zeros((*B, D), device="cuda")
    hs = ttm.glr_step(x, g, state)
    close(flat(hs), rh, th, x.dtype)


def test_no_tokens_returns_the_state():
    s = torch.randn(3, 16, device="cuda")
    x = torch.empty(3, 0, 16, device="cuda")
    h, last = ttm.glr_fwd(x, x, h0=s)
    assert h.shape == (3, 0, 16) and torch.equal(last, s)
    assert not ttm.glr_fwd(x, x)[1].any()
    out = ttm.glr_bwd(x, h, x, h0=s, dh_last=s)
    assert torch.equal(out["dh0"], s) and out["dg"].shape == (3, 0, 16)


@pytest.mark.parametrize("token", [False, True])
def test_reset_hides_what_is_before_it(token):
    """Nothing before a token with g = -inf reaches it or later ones, nor their gradient back."""
    x, g, h0 = make(2, 400, 32, "f32", token, seed=5)
    g[:, 250] = -math.inf
    a, _ = ttm.glr_fwd(on(x), on(g), h0=on(h0))
    b, _ = ttm.glr_fwd(on(x[:, 250:]), on(g[:, 250:]))
    rh, th, _, _ = reference(x, g, h0)
    close(a, rh, th, torch.float32)
    close(b, rh[:, 250:], th[:, 250:], torch.float32)
    dh = torch.ones_like(x)
    out = ttm.glr_bwd(on(g), a, on(dh), h0=on(h0))
    assert not out["dg"][:, 250].any()


@pytest.mark.parametrize("token", [False, True])
def test_gradient_against_differences(token):
    """dL for L = <dh, h> + <dh_last, h_last>, by central differences of the float64 loop:
    the step 1e-5 leaves about 1e-9, so fp32's own error decides (rel 1e-5 of the largest)."""
    N, T, D = 1, 37, 5
    x, g, h0 = make(N, T, D, "f32", token, seed=9)
    r = torch.Generator().manual_seed(2)
    dh, dl = torch.randn((N, T, D), generator=r), torch.randn((N, D), generator=r)

    def loss(x, g, h0):
        a, h, L = torch.exp(g), h0, 0.0
        a = a if a.dim() == 3 else a[..., None]
        for t in range(T):
            h = a[:, t] * h + x[:, t]
            L = L + (dh[:, t].double() * h).sum()
        return float(L + (dl.double() * h).sum())

    h = reference(x, g, h0)[0].float()
    out = ttm.glr_bwd(on(g), on(h), on(dh), h0=on(h0), dh_last=on(dl))
    args = [x.double(), g.double(), h0.double()]
    for k, name in enumerate(("dx", "dg", "dh0")):
        diff = torch.empty_like(args[k]).reshape(-1)
        for i in range(diff.numel()):
            v = []
            for e in (1e-5, -1e-5):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += e
                v.append(loss(*moved))
            diff[i] = (v[0] - v[1]) / 2e-5
        got = out[name].double().cpu().reshape(-1)
        assert float((got - diff).abs().max()) < 1e-5 * float(diff.abs().max()), name


def test_another_stream_and_given_outputs():
    x, g, h0 = (on(t) for t in make(4, 3000, 128, "bf16", False))
    want, want_last = ttm.glr_fwd(x, g, h0=h0)
    h, last = torch.empty_like(want), torch.empty_like(want_last)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got, got_last = ttm.glr_fwd(x, g, h0=h0, h=h, h_last=last, stream=s)
    s.synchronize()
    assert got is h and torch.equal(h, want) and torch.equal(got_last, want_last)


@pytest.mark.parametrize("T,D,N", [(5000, 128, 2), (40000, 64, 1), (333, 16, 700)])
def test_captured_in_a_graph(T, D, N):
    x, g, h0 = (on(t) for t in make(N, T, D, "bf16", False))
    want, _ = ttm.glr_fwd(x, g, h0=h0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, _ = ttm.glr_fwd(x, g, h0=h0)
        d = ttm.glr_bwd(g, h, x, h0=h0)
    for _ in range(3):
        h.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)
    ref = ttm.glr_bwd(g, want, x, h0=h0)
    assert all(torch.equal(d[k], ref[k]) for k in d)


def test_refusals():
    x = torch.randn(2, 10, 16, device="cuda")
    g = torch.zeros_like(x)
    bad = [lambda: ttm.glr_fwd(x, g[:, :9]), lambda: ttm.glr_fwd(x, g.bfloat16()),
           lambda: ttm.glr_fwd(x, g[..., 0].bfloat16()), lambda: ttm.glr_fwd(x[..., ::2], g[..., ::2]),
           lambda: ttm.glr_fwd(x, g, h0=torch.zeros(2, 15, device="cuda")),
           lambda: ttm.glr_fwd(x, g, h0=torch.zeros(2, 16, device="cuda", dtype=torch.float64)),
           lambda: ttm.glr_fwd(x, g, h=x), lambda: ttm.glr_fwd(x, g.cpu()),
           lambda: ttm.glr_fwd(x, g, h=torch.empty(2, 10, 17, device="cuda")),
           lambda: ttm.glr_fwd(x.expand(2, 10, 16)[:1].expand(3, 10, 16), g[:1].expand(3, 10, 16)),
           lambda: ttm.glr_bwd(g, x[:, :9], x), lambda: ttm.glr_bwd(g, x, x, out=dict(dx=x)),
           lambda: ttm.glr_step(x, g, None), lambda: ttm.glr_step(x[:, :0], g[:, :0], torch.zeros(2, 16, device="cuda")),
           lambda: ttm.glr_step(x, g, torch.zeros(2, 16, device="cuda").bfloat16())]
    for f in bad:
        with pytest.raises(ttm.TTMError) as e:
            f()
        assert e.value.code == ttm.ERR_INVALID_ARG
    with pytest.raises(TypeError):
        ttm.glr_fwd(x.half(), g.half())


@pytest.mark.parametrize("N,T,D", [(1, 16, 64), (2, 10, 36), (3, 15, 7), (300, 18, 70), (64, 48, 768),
                                   (160, 21, 1001), (160, 130, 1001), (2500, 3, 512), (2500, 7, 512),
                                   (3000, 2, 44)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("token,pad", [(False, 0), (False, 3), (True, 0)])
def test_short_sequences_and_many_channels(N, T, D, dtype, token, pad):
    x, g, h0 = make(N, T, D, dtype, token, seed=N + T, resets=True)
    dh = make(N, T, D, dtype, True, seed=N + T + 1)[0]

    def view(t):
        wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), math.nan, dtype=t.dtype, device="cuda")
        wide[..., :t.shape[-1]] = t.cuda()
        return wide[..., :t.shape[-1]]

    xc, gc, dhc = view(x), (view(g) if not token else g.cuda()), view(dh)
    h, last = ttm.glr_fwd(xc, gc, h0=on(h0))
    rh, th, rl, tl = reference(x, g, h0)
    close(h, rh, th, x.dtype)
    close(last, rl, tl, torch.float32)
    rh = rh.to(x.dtype)
    out = ttm.glr_bwd(gc, on(rh), dhc, h0=on(h0))
    dx, tx, dg, tg, c, tc = grad_reference(g, rh, h0, dh, None)
    close(out["dx"], dx, tx, x.dtype)
    close(out["dg"], dg, tg, g.dtype)
    close(out["dh0"], c, tc, torch.float32)


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("T,D", [(6, 64), (40, 64), (300, 64), (2500, 8)])
def test_gates_far_from_zero(token, T, D):
    """The bound holds however far a gate is from 0: states decay from 1e37 through gates of -30 to -1
    and are brought back by a value of 1e30 now and then.  The retention over a stretch of tokens is a product
    that goes to 0 below 2^-126, so a state errs by that share of the largest one before it too."""
    r = torch.Generator().manual_seed(T)
    shape = (40, T) if token else (40, T, D)
    x = torch.zeros((40, T, D))
    x[:, ::9] = 1e30 * torch.randn((40, (T + 8) // 9, D), generator=r)
    g = -torch.exp(math.log(30.0) * torch.rand(shape, generator=r))
    h0 = 1e37 * torch.randn((40, D), generator=r)
    h, last = ttm.glr_fwd(on(x), on(g), h0=on(h0))
    rh, th, rl, tl = reference(x, g, h0)
    lost = 2.0 ** -126 * max(float(h0.abs().max()), float(rh.abs().max()))
    close(h, rh, th + lost, torch.float32)
    close(last, rl, tl + lost, torch.float32)
    rh = rh.float()
    out = ttm.glr_bwd(on(g), on(rh), on(x), h0=on(h0 * 1e-30), dh_last=on(h0))
    dx, _, dg, _, c, _ = grad_reference(g, rh, h0 * 1e-30, x, h0)
    assert all(bool(torch.isfinite(t).all()) for t in (out["dx"], out["dh0"]))
    _, tx, _, _, _, tc = grad_reference(g, rh, h0 * 1e-30, x, h0)
    close(out["dx"], dx, tx + lost, torch.float32)
    close(out["dh0"], c, tc + lost, torch.float32)


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("T,D,dtype", [(100, 8, "f32"), (2000, 4, "f32"), (3900, 4, "bf16"), (5000, 64, "f32"),
                                       (3000, 131, "bf16")])
def test_growing_gates(token, T, D, dtype):
    """A state of 1e-30 that grows by e^130 in all, one more than fp32 holds, before a reset and after it:
    every state is finite although the retention over such a stretch is not."""
    r = torch.Generator().manual_seed(T)
    shape = (3, T) if token else (3, T, D)
    g = (240.0 / T) * (1 + 0.1 * torch.rand(shape, generator=r))
    g[:, T // 2] = -math.inf
    g = g.to(torch.float32 if token else DT[dtype])
    x = torch.zeros((3, T, D), dtype=DT[dtype])
    x[:, T // 2] = 1e-30
    x[:, T // 2 + 1] = 1e-30 * torch.randn((3, D), generator=r)
    h0 = 1e-30 * torch.randn((3, D), generator=r)
    h, last = ttm.glr_fwd(on(x), on(g), h0=on(h0))
    rh, th, rl, tl = reference(x, g, h0)
    assert float(rh.abs().max()) > 1e20
    close(h, rh, th, x.dtype)
    close(last, rl, tl, torch.float32)
    dh, dl = torch.zeros_like(x), 1e-30 * torch.randn((3, D), generator=r)
    rh = torch.ones_like(x)
    out = ttm.glr_bwd(on(g), on(rh), on(dh), h0=on(h0), dh_last=on(dl))
    dx, tx, dg, tg, c, tc = grad_reference(g, rh, h0, dh, dl)
    close(out["dx"], dx, tx, x.dtype)
    close(out["dg"], dg, tg, g.dtype)
    close(out["dh0"], c, tc, torch.float32)


@pytest.mark.parametrize("N,T,D", [(3, 700, 64), (16, 40, 136), (5, 1025, 16), (2, 3000, 131), (1, 600, 64), (300, 9, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["time first", "padded sequences", "windows", "mixed"])
@pytest.mark.parametrize("token", [False, True])
def test_other_orders(N, T, D, dtype, order, token):
    """Tokens further apart than sequences, sequences a stride apart that no number of tokens makes, windows that
    share their rows, and x and g of two orders: the results are those of contiguous tensors, bit for bit."""
    x, g, h0 = (on(t) for t in make(N, T, D, dtype, token, seed=N + T, resets=True))
    if token and dtype == "bf16":
        g = g.float()

    def lay(t, how):
        if how == "time first":
            return t.transpose(0, 1).contiguous().transpose(0, 1)
        inner = t[0].numel()
        if how == "padded sequences":                 # 24 or 8 elements: rows stay on 16 bytes, or do not
            buf = torch.full((N, inner + (24 if D % 8 == 0 else 8)), math.nan, dtype=t.dtype, device="cuda")
            v = buf[:, :inner].view(N, *t.shape[1:]) if N == 1 else buf.as_strided(
                t.shape, (buf.stride(0), *t[0].stride()))
        else:                                         # windows: sequence n starts at token n of the first
            row = t[0, 0].numel()
            buf = torch.cat((t[0].reshape(T, row), t[:N, -1].reshape(N, row)))
            return buf.as_strided(t.shape, (row, *t[0].stride()))
        v.copy_(t)
        return v

    xo = lay(x, "time first" if order == "mixed" else order)
    go = lay(g, "padded sequences" if order == "mixed" else order)
    h, last = ttm.glr_fwd(xo, go, h0=h0)
    xc, gc = xo.contiguous(), go.contiguous()
    rh, th, rl, tl = reference(xc.cpu(), gc.cpu(), h0.cpu())
    close(h, rh, th, x.dtype)
    close(last, rl, tl, torch.float32)
    out, same = ttm.glr_bwd(go, h, xo, h0=h0), ttm.glr_bwd(gc, h, xc, h0=h0)
    assert torch.equal(ttm.glr_fwd(xc, gc, h0=h0)[0], h)
    dx, tx, dg, tg, c, tc = grad_reference(gc.cpu(), h.cpu(), h0.cpu(), xc.cpu(), None)
    close(out["dx"], dx, tx, x.dtype)
    close(out["dg"], dg, tg, g.dtype)
    close(out["dh0"], c, tc, torch.float32)
    assert all(torch.equal(out[k], same[k]) for k in out)
    if T < 50:
        state = h0.clone()
        assert torch.equal(ttm.glr_step(xo, go, state), ttm.glr_step(xc, gc, h0.clone()))
