"""Gated feed-forward block and its gradient against float64.

Tolerances, elementwise.  A product over K terms with fp32 sums errs by at most k(K) = (K + 64) 2^-24 of the sum of
sizes (the tensor cores cut a sum of 16 products and the running one off at 2^-22 of the largest: K / 4 in
these units).  act and its slope add 2^-20 of themselves (erf and exponentials of a few units, |g| 2^-24 more)
and carry an error of g on times 1.2 (slope at most 1.13; second derivative at most 0.8).  h, dg and du are rounded to
bf16 (2^-8 of themselves) before the next product, and so is the result.  These bounds add up sizes, so the norm
of the error is held as well, where there are values enough: two independent roundings of 2^-8 at most, uniform
within a step, come to 2.4e-3; 2^-8 is the bound."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
BF, U, HALF = torch.bfloat16, 2.0 ** -24, 2.0 ** -8
ACT = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def near(got, ref, tol, name=""):
    got = got.detach().double()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol + HALF * (ref.abs() + tol) + 1e-37)
    assert not bad.any(), (name, int(bad.sum()), float((got - ref).abs().max()), bad.nonzero()[:4].tolist())
    if got.numel() >= 4096:
        assert float((got - ref).norm()) <= HALF * float(ref.norm()), (name, float((got - ref).norm() / ref.norm()))


def k(n):
    return (n + 64) * U


def make(N, D, F, seed=0, pad=0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=r, device="cuda")  # noqa: E731
    x, dy, res = (rand(N, D + pad).to(BF)[:, :D] for _ in range(3))
    return x, dy, res, (rand(D, 2 * F) / D ** 0.5).to(BF), (rand(F, D) / F ** 0.5).to(BF)


def act64(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = 0.5 * torch.erfc(-g / 2 ** 0.5)
    return g * c, c + g * torch.exp(-0.5 * g * g) / (2 * torch.pi) ** 0.5


def check(N, D, F, act="silu", residual=True, pad=0, seed=0, grad=True):
    x, dy, res, W_in, W_out = make(N, D, F, seed, pad)
    x64, y64, A, B = (t.double() for t in (x, dy, W_in, W_out))
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out, act=act, residual=res if residual else None)
    ref = x64 @ A
    tg = k(D) * (x64.abs() @ A.abs())
    near(gu, ref, tg, "gu")
    g, u, eg, eu = ref[:, :F], ref[:, F:], tg[:, :F], tg[:, F:]
    a, _ = act64(g, act)
    h = a * u
    eh = 1.2 * eg * (u.abs() + eu) + a.abs() * eu + ACT * h.abs()
    eh = eh + HALF * (h.abs() + eh)
    want, tol = h @ B, (eh + k(F) * h.abs()) @ B.abs()
    if residual:
        want, tol = want + res.double(), tol + U * want.abs()
    near(y, want, tol, "y")
    only, none = ttm.gated_ffn_fwd(x, W_in, W_out, act=act, residual=res if residual else None, want_gu=False)
    assert none is None and torch.equal(only, y)
    if not grad:
        return
    call = lambda **o: ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out, act=act, **o)  # noqa: E731
    d = call()
    g, u = gu[:, :F].double(), gu[:, F:].double()       # the gradient takes them as they were written
    a, slope = act64(g, act)
    dh, eh = y64 @ B.T, k(D) * (y64.abs() @ B.abs().T)
    dgu = torch.cat((dh * u * slope, dh * a), 1)
    e = torch.cat((eh * (u * slope).abs(), eh * a.abs()), 1) + ACT * (dgu.abs() + torch.cat(((dh * u).abs(), dgu[:, F:].abs()), 1))
    e = e + HALF * (dgu.abs() + e)
    near(d["dx"], dgu @ A.T, (e + k(2 * F) * dgu.abs()) @ A.abs().T, "dx")
    near(d["dW_in"], x64.T @ dgu, x64.abs().T @ (e + k(N) * dgu.abs()), "dW_in")
    h = a * u
    near(d["dW_out"], h.T @ y64, ((HALF + ACT + k(N)) * h.abs()).T @ y64.abs(), "dW_out")
    again = call()
    assert all(torch.equal(d[n], again[n]) for n in d)
    part = call(want_dw=False)
    assert part["dW_in"] is None and torch.equal(part["dx"], d["dx"])
    part = call(want_dx=False)
    assert part["dx"] is None and torch.equal(part["dW_in"], d["dW_in"]) and torch.equal(part["dW_out"], d["dW_out"])


@pytest.mark.parametrize("N", [1, 2, 7, 16, 33, 64, 65, 100, 128, 129, 200, 256, 257, 500])
@pytest.mark.parametrize("D,F", [(8, 8), (64, 128), (72, 264), (256, 1000), (520, 328)])
def test_sizes(N, D, F):
    check(N, D, F, act="gelu" if N % 2 else "silu", residual=N % 3 != 0, pad=8 * (N % 2), seed=N)


@pytest.mark.parametrize("N,D,F", [(1, 2048, 5504), (16, 2048, 5504), (48, 768, 2048), (300, 2048, 512), (1537, 768, 2056),
                                   (777, 1000, 3000), (2048, 512, 1024), (4097, 136, 72), (1000, 24, 4096), (130, 4096, 40),
                                   (5000, 1032, 776), (9001, 264, 2008), (20011, 520, 136), (2300, 2048, 2816),
                                   (330, 2048, 5504), (250, 2048, 5504), (500, 768, 2048), (768, 136, 2048), (769, 136, 2048),
                                   (640, 2048, 1544), (385, 520, 5504)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_larger(N, D, F, act):
    check(N, D, F, act)


def test_leading_dimensions_and_strides():
    x, dy, res, W_in, W_out = make(60, 64, 96)
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out, residual=res)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)
    wide = torch.randn(60, 200, device="cuda").to(BF)
    xs, rs, ds = wide[:, 8:72], torch.empty(60, 72, device="cuda", dtype=BF)[:, :64], wide.clone()[:, 64:128]
    xs.copy_(x), rs.copy_(res), ds.copy_(dy)
    y2, gu2 = ttm.gated_ffn_fwd(xs, W_in, W_out, residual=rs)
    assert torch.equal(y2, y) and torch.equal(gu2, gu)
    d2 = ttm.gated_ffn_bwd(ds, xs, gu, W_in, W_out)
    assert all(torch.equal(d[n], d2[n]) for n in d)
    y3, gu3 = ttm.gated_ffn_fwd(x.view(3, 4, 5, 64), W_in, W_out, residual=res.view(3, 4, 5, 64))
    assert torch.equal(y3.view(60, 64), y) and gu3.shape == (3, 4, 5, 192)


def test_no_rows():
    x, _, _, W_in, W_out = make(3, 64, 96)
    y, gu = ttm.gated_ffn_fwd(x[:0], W_in, W_out)
    assert y.shape == (0, 64) and gu.shape == (0, 192)
    d = ttm.gated_ffn_bwd(x[:0], x[:0], gu, W_in, W_out)
    assert d["dx"].shape == (0, 64) and not d["dW_in"].any() and not d["dW_out"].any()


@pytest.mark.parametrize("N", [5, 300, 900])
def test_values_that_are_not_finite_stay_in_their_row(N):
    x, dy, res, W_in, W_out = make(N, 128, 256)
    want, gu = ttm.gated_ffn_fwd(x, W_in, W_out, residual=res)
    bad = x.clone()
    bad[2, 5] = float("nan")
    bad[4, 7] = float("inf")
    y, _ = ttm.gated_ffn_fwd(bad, W_in, W_out, residual=res)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[2] = keep[4] = False
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_far_from_zero(act):
    """act and its slope where exponentials overflow or vanish."""
    g = torch.tensor([-1e4, -300.0, -90.0, -30.0, -9.0, -1.0, 0.0, 1.0, 9.0, 30.0, 90.0, 300.0, 1e4, -88.0, 88.0, 4.0]).to(BF)
    D = 16
    gu = torch.cat((g, torch.ones(16, dtype=BF)))[None].cuda()
    eye = torch.eye(16, dtype=BF, device="cuda")
    W_in = torch.cat((eye, eye), 1)
    a, slope = act64(g.double().cuda(), act)
    d = ttm.gated_ffn_bwd(torch.ones(1, D, device="cuda", dtype=BF), torch.zeros(1, D, device="cuda", dtype=BF), gu, W_in, eye, act=act)
    near(d["dx"], (slope + a)[None], 1e-6 + 2 * HALF * (slope.abs() + a.abs())[None])
    x = g[None].cuda()
    y, _ = ttm.gated_ffn_fwd(x, torch.cat((eye, torch.zeros_like(eye)), 1), eye, act=act)
    assert torch.isfinite(y).all() and not y.any()      # act(g) times u = 0
    near(ttm.gated_ffn_bwd(eye, eye, torch.cat((g.expand(16, 16), torch.ones(16, 16)), 1).to(BF).cuda(), W_in, eye, act=act)["dW_out"],
         a[:, None].expand(16, 16), 1e-30 + HALF * a.abs()[:, None])


def test_gradient_against_differences():
    """Along whole directions of x, W_in and W_out, central differences in float64 of <dy, y>; the gradient's three
    roundings of 2^-8 at most, over hundreds of values, stay below 2^-7 of the sizes' norm."""
    x, dy, _, W_in, W_out = make(20, 32, 48, seed=3)
    _, gu = ttm.gated_ffn_fwd(x, W_in, W_out)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)

    def loss(x, A, B):
        g = x @ A
        return float((dy.double() * ((act64(g[:, :48], "silu")[0] * g[:, 48:]) @ B)).sum())
    args = [t.double() for t in (x, W_in, W_out)]
    for i, n in enumerate(("dx", "dW_in", "dW_out")):
        v = torch.randn_like(args[i])
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - 1e-5 * v, args[i] + 1e-5 * v
        want = (loss(*hi) - loss(*lo)) / 2e-5
        got = float((d[n].double() * v).sum())
        assert abs(got - want) < 2.0 ** -7 * float(d[n].double().norm() * 3), (n, got, want)


def test_offsets_past_32_bits():
    """gu of 2.2e9 values: the last rows as a call on them alone gives them (other tiles, so within the roundings)."""
    N, D, F = 200003, 64, 5504
    x, dy, res, W_in, W_out = make(N, D, F)
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out, residual=res)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out, want_dw=False)
    tail = [t[-300:].contiguous() for t in (x, dy, res)]
    y2, gu2 = ttm.gated_ffn_fwd(tail[0], W_in, W_out, residual=tail[2])
    d2 = ttm.gated_ffn_bwd(tail[1], tail[0], gu[-300:].contiguous(), W_in, W_out, want_dw=False)
    for a, b in ((y[-300:], y2), (gu[-300:], gu2), (d["dx"][-300:], d2["dx"])):
        assert float((a.double() - b.double()).norm()) <= HALF * float(b.double().norm())


@pytest.mark.parametrize("N", [9, 400, 1100])
def test_streams_graphs_and_given_outputs(N):
    x, dy, res, W_in, W_out = make(N, 256, 512)
    y, gu = ttm.gated_ffn_fwd(x, W_in, W_out, residual=res)
    d = ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, gu2 = ttm.gated_ffn_fwd(x, W_in, W_out, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(y2, y) and torch.equal(gu2, gu)
    out = {n: torch.zeros_like(t) for n, t in d.items()}
    y2, gu2 = torch.zeros_like(y), torch.zeros_like(gu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ttm.gated_ffn_fwd(x, W_in, W_out, residual=res, y=y2, gu=gu2)
        ttm.gated_ffn_bwd(dy, x, gu2, W_in, W_out, out=out)
    for _ in range(2):
        y2.zero_(), gu2.zero_(), [t.zero_() for t in out.values()]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(gu2, gu) and all(torch.equal(out[n], d[n]) for n in d)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, give the bits of calls one by one."""
    a, b = make(700, 512, 1024, seed=1), make(40, 512, 1024, seed=2)
    want = [ttm.gated_ffn_fwd(t[0], t[3], t[4])[0] for t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (s, t) in enumerate(zip(streams, (a, b))):
            got[i].append(ttm.gated_ffn_fwd(t[0], t[3], t[4], stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_refusals():
    x, dy, res, W_in, W_out = make(10, 64, 96)
    gu = ttm.gated_ffn_fwd(x, W_in, W_out)[1]
    odd = torch.zeros(10, 68, device="cuda", dtype=BF)[:, 4:]           # rows not on 16 bytes
    bad = [lambda: ttm.gated_ffn_fwd(x, W_in, W_out, act="relu"), lambda: ttm.gated_ffn_fwd(odd, W_in, W_out),
           lambda: ttm.gated_ffn_fwd(x, W_in, W_out, residual=odd), lambda: ttm.gated_ffn_fwd(x, W_in, W_out, residual=res[:9]),
           lambda: ttm.gated_ffn_fwd(x, W_in[:, :190], W_out), lambda: ttm.gated_ffn_fwd(x, W_in, W_out[:95]),
           lambda: ttm.gated_ffn_fwd(x, W_in.float(), W_out), lambda: ttm.gated_ffn_fwd(x.cpu(), W_in, W_out),
           lambda: ttm.gated_ffn_fwd(x[:, :60], W_in[:60].contiguous(), W_out[:, :60].contiguous()),
           lambda: ttm.gated_ffn_fwd(x, W_in, W_out, y=x), lambda: ttm.gated_ffn_fwd(x, W_in, W_out, residual=res, y=res),
           lambda: ttm.gated_ffn_bwd(dy, x, gu[:, :96], W_in, W_out), lambda: ttm.gated_ffn_bwd(dy[:9], x, gu, W_in, W_out),
           lambda: ttm.gated_ffn_bwd(odd, x, gu, W_in, W_out), lambda: ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out, out=dict(dx=dy)),
           lambda: ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out, workspace=torch.empty(16, device="cuda"))]
    for call in bad:
        with pytest.raises(ttm.TTMError):
            call()
    with pytest.raises(TypeError):
        ttm.gated_ffn_fwd(x.float(), W_in.float(), W_out.float())
