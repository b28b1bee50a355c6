"""Layer norm and its gradient against float64.

Tolerances, elementwise.  A sum of D values by threads that take up to D / 8 of them each and
join by halves errs by at most q = (D / 8 + 12) 2^-24 of the sum of sizes.  So the mean is off
by em = q mean|x|, the variance by a share of about q + 2^-22 plus em^2 (rstd by half of that
share), and (x - mean) rstd by rstd em + |n| (q / 2 + 2^-22).  The gradient's two means err by q
of the mean of sizes, and everything by a few units more.  A bf16 result (8 significant bits) adds 2^-8 of itself."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def close(got, ref, tol, dtype=torch.float32):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape
    bad = (got - ref).abs() > tol + HALF[dtype] * (ref.abs() + tol) + 1e-37
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


def make(N, D, dtype, affine, pad=0, seed=0):
    r = torch.Generator().manual_seed(seed)
    wide = torch.randn((N, D + pad), generator=r).to(DT[dtype])
    wide += torch.randn((D + pad,), generator=r).to(DT[dtype])
    w = 1 + 0.2 * torch.randn((D,), generator=r) if affine else None
    b = torch.randn((D,), generator=r) if affine else None
    dy = torch.randn((N, D + pad), generator=r).to(DT[dtype])
    return wide, w, b, dy


def stats(x, eps):
    mean = x.mean(-1)
    return mean, 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)


SHAPES = [(1, 1), (3, 2), (1, 64), (7, 64), (1000, 64), (33, 128), (5, 199), (64, 768), (9, 1000),
          (130, 2048), (4, 3001), (3, 4096), (2, 8192), (2, 16384), (1, 20011), (1, 40000),
          (4099, 24), (20000, 8)]


@pytest.mark.parametrize("N,D", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("affine,pad", [(True, 0), (False, 0), (True, 8), (False, 3)])
def test_forward_and_gradient(N, D, dtype, affine, pad):
    wide, w, b, dyw = make(N, D, dtype, affine, pad, seed=N + D)
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    x = on(wide)[:, :D]
    dt, eps = DT[dtype], 1e-5
    y, mean, rstd = ttm.layer_norm_fwd(x, on(w), on(b), eps=eps)
    f = wide[:, :D].double()
    rm, rr = stats(f, eps)
    q = (D / 8 + 12) * 2.0 ** -24
    em = q * f.abs().mean(-1) + 2.0 ** -24 * rm.abs()
    n = (f - rm[:, None]) * rr[:, None]
    share = q + 2.0 ** -22 + em ** 2 * rr ** 2
    close(mean, rm, em)
    close(rstd, rr, rr * (share / 2 + 2.0 ** -22))
    tn = (rr * em)[:, None] + n.abs() * (share / 2 + 2.0 ** -21)[:, None]
    ref = n * w.double() + b.double() if affine else n
    size = w.double().abs() if affine else torch.ones(D, dtype=torch.float64)
    close(y, ref, tn * size + 2.0 ** -23 * ((n * size).abs() + (b.double().abs() if affine else 0)), dt)

    # the gradient takes the forward's statistics as they were written
    dy = on(dyw)[:, :D]
    out = ttm.layer_norm_bwd(dy, x, mean, rstd, on(w))
    m64, r64 = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    n, g = (f - m64) * r64, dyw[:, :D].double()
    u = g * size * (torch.sign(w.double()) if affine else 1)
    en = 2.0 ** -23 * (n.abs() + (m64 * r64).abs())      # rounding of (x - mean) rstd
    s1, s2 = u.mean(-1, keepdim=True), (u * n).mean(-1, keepdim=True)
    t1 = (q + 2.0 ** -23) * u.abs().mean(-1, keepdim=True)
    t2 = (q + 2.0 ** -22) * (u * n).abs().mean(-1, keepdim=True) + (u.abs() * en).mean(-1, keepdim=True)
    dx = r64 * (u - s1 - n * s2)
    tol = r64 * (t1 + n.abs() * t2 + en * s2.abs() + 2.0 ** -21 * (u.abs() + s1.abs() + (n * s2).abs()))
    close(out["dx"], dx, tol, dt)
    rows = (N + 12) * 2.0 ** -24
    close(out["db"], g.sum(0), rows * g.abs().sum(0))
    close(out["dw"], (g * n).sum(0), (rows + 2.0 ** -22) * (g * n).abs().sum(0) + (g.abs() * en).sum(0))
    again = ttm.layer_norm_bwd(dy, x, mean, rstd, on(w))
    assert all(torch.equal(out[k], again[k]) for k in out)
    part = ttm.layer_norm_bwd(dy, x, mean, rstd, on(w), want_db=False)
    assert part["db"] is None and torch.equal(part["dw"], out["dw"]) and torch.equal(part["dx"], out["dx"])
    none = ttm.layer_norm_bwd(dy, x, mean, rstd, on(w), want_db=False, want_dw=False)
    assert none["dw"] is None and torch.equal(none["dx"], out["dx"])


def test_large_mean_keeps_the_variance():
    """Rows at 1e4 with a spread of one: sums of squares about zero would lose it."""
    r = torch.Generator().manual_seed(0)
    x = 1e4 + torch.randn((5, 4096), generator=r)
    y, mean, rstd = ttm.layer_norm_fwd(x.cuda(), eps=0.0)
    rm, rr = stats(x.double(), 0.0)
    em = (4096 / 8 + 12) * 2.0 ** -24 * 1e4
    assert float((rstd.double().cpu() / rr - 1).abs().max()) < em ** 2 / 2 + 1e-4
    assert float((mean.double().cpu() - rm).abs().max()) < em


def test_constant_rows_and_eps():
    x = torch.full((3, 100), 2.5, device="cuda")
    y, mean, rstd = ttm.layer_norm_fwd(x, eps=1e-4)
    assert not y.any() and bool((mean == 2.5).all())
    assert float((rstd - 100).abs().max()) < 1e-4


def test_leading_dimensions_and_empty():
    x = torch.randn(2, 5, 3, 40, device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn(40, device="cuda"), torch.randn(40, device="cuda")
    y, mean, rstd = ttm.layer_norm_fwd(x, w, b)
    y2, m2, r2 = ttm.layer_norm_fwd(x.reshape(-1, 40), w, b)
    assert torch.equal(y.reshape(-1, 40), y2) and mean.shape == (2, 5, 3)
    e = x[:0]
    y, mean, rstd = ttm.layer_norm_fwd(e, w, b)
    out = ttm.layer_norm_bwd(e, e, mean, rstd, w)
    assert y.shape == e.shape and not out["dw"].any() and not out["db"].any()
    y, mean, rstd = ttm.layer_norm_fwd(x, w, b, want_stats=False)
    assert mean is None and torch.equal(y.reshape(-1, 40), y2)


def test_gradient_against_differences():
    """dL of L = <dy, y> by central differences in float64 (step 1e-5, error about 1e-9)."""
    r = torch.Generator().manual_seed(4)
    x, w = torch.randn((3, 7), generator=r), torch.randn((7,), generator=r)
    b, dy = torch.randn((7,), generator=r), torch.randn((3, 7), generator=r)

    def loss(x, w, b):
        m, s = stats(x, 1e-5)
        return float((dy.double() * ((x - m[:, None]) * s[:, None] * w + b)).sum())

    _, mean, rstd = ttm.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    out = ttm.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    args = [x.double(), w.double(), b.double()]
    for k, name in enumerate(("dx", "dw", "db")):
        diff = torch.empty(args[k].numel(), dtype=torch.float64)
        for i in range(diff.numel()):
            v = []
            for e in (1e-5, -1e-5):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += e
                v.append(loss(*moved))
            diff[i] = (v[0] - v[1]) / 2e-5
        got = out[name].double().cpu().reshape(-1)
        assert float((got - diff).abs().max()) < 1e-5 * max(1.0, float(diff.abs().max())), name


def test_refusals():
    x = torch.randn(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    y, mean, rstd = ttm.layer_norm_fwd(x, w, w)
    bad = [lambda: ttm.layer_norm_fwd(x, w[:15]), lambda: ttm.layer_norm_fwd(x, w.bfloat16()),
           lambda: ttm.layer_norm_fwd(x[:, ::2]), lambda: ttm.layer_norm_fwd(x, y=x),
           lambda: ttm.layer_norm_fwd(x, eps=-1.0), lambda: ttm.layer_norm_fwd(x, eps=float("nan")),
           lambda: ttm.layer_norm_fwd(x.cpu()), lambda: ttm.layer_norm_fwd(x[:1].expand(4, 16)),
           lambda: ttm.layer_norm_bwd(x[:3], x, mean, rstd), lambda: ttm.layer_norm_bwd(x, x, None, rstd),
           lambda: ttm.layer_norm_bwd(x.bfloat16(), x, mean, rstd),
           lambda: ttm.layer_norm_bwd(x, x, mean, rstd, out=dict(dx=x)),
           lambda: ttm.layer_norm_bwd(x, x, mean[:3], rstd),
           lambda: ttm.layer_norm_bwd(x, x, mean, rstd, workspace=torch.empty(4, device="cuda"))]
    for f in bad:
        with pytest.raises(ttm.TTMError) as e:
            f()
        assert e.value.code == ttm.ERR_INVALID_ARG
    with pytest.raises(TypeError):
        ttm.layer_norm_fwd(x.half())


@pytest.mark.parametrize("N,D", [(70, 3), (70, 12), (300, 16), (70, 24), (70, 32), (70, 96), (70, 131), (70, 300),
                                 (70, 500), (70, 513), (330, 771), (330, 600), (40, 1026), (40, 1600), (40, 2050),
                                 (20, 3074), (20, 4098), (700, 6000), (330, 8184), (700, 12000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 3, 1, 2, 4])
def test_row_lengths_and_starts(N, D, dtype, pad):
    test_forward_and_gradient(N, D, dtype, pad != 1, pad)


@pytest.mark.parametrize("D", [131, 300, 500, 513, 771, 900, 1026])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1])
def test_many_rows(D, dtype, pad):
    test_forward_and_gradient(4100, D, dtype, True, pad)


@pytest.mark.parametrize("N,D", [(40, 64), (70, 131), (33, 768), (9, 1000), (130, 2048), (5, 8192), (5000, 300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [1e3, 1e4])
def test_gradient_of_rows_far_from_zero(N, D, dtype, at):
    """For the given statistics n = (x - mean) rstd errs by two roundings, 2^-23 of itself, however large
    the mean is against the spread; the other bounds as in test_forward_and_gradient."""
    wide, w, _, dy = make(N, D, dtype, True, seed=N + D)
    x = (at + (4.0 if dtype == "f32" else at / 8) * wide.float()).to(DT[dtype])
    mean, rstd = (t.float() for t in stats(x.double(), 1e-5))
    out = ttm.layer_norm_bwd(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), w.cuda())
    m64, r64 = mean.double()[:, None], rstd.double()[:, None]
    q = (D / 8 + 12) * 2.0 ** -24
    n, g = (x.double() - m64) * r64, dy.double()
    u, en = g * w.double(), 2.0 ** -23 * n.abs()
    s1, s2 = u.mean(-1, keepdim=True), (u * n).mean(-1, keepdim=True)
    t1 = (q + 2.0 ** -23) * u.abs().mean(-1, keepdim=True)
    t2 = (q + 2.0 ** -22) * (u * n).abs().mean(-1, keepdim=True) + (u.abs() * en).mean(-1, keepdim=True)
    tol = r64 * (t1 + n.abs() * t2 + en * s2.abs() + 2.0 ** -21 * (u.abs() + s1.abs() + (n * s2).abs()))
    close(out["dx"], r64 * (u - s1 - n * s2), tol, DT[dtype])
    rows = (N + 12) * 2.0 ** -24
    close(out["dw"], (g * n).sum(0), (rows + 2.0 ** -22) * (g * n).abs().sum(0) + (g.abs() * en).sum(0))
    close(out["db"], g.sum(0), rows * g.abs().sum(0))


@pytest.mark.parametrize("D", [24, 64, 100, 131, 771, 1000, 2048, 3001, 20011])
@pytest.mark.parametrize("value", [100.0, 1e36, 3e38])
def test_gradient_of_constant_rows(D, value):
    """x = mean everywhere, so n = 0: dw = 0 and dx = rstd (u - mean u), also where mean rstd is past fp32."""
    r = torch.Generator().manual_seed(1)
    x, dy = torch.full((6, D), value), torch.randn((6, D), generator=r)
    mean, rstd = torch.full((6,), value), torch.full((6,), 1e-5 ** -0.5)
    out = ttm.layer_norm_bwd(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda())
    assert not out["dw"].any()
    u, r64 = dy.double(), rstd.double()[:, None]
    q = (D / 8 + 12) * 2.0 ** -24
    s1 = u.mean(-1, keepdim=True)
    tol = r64 * ((q + 2.0 ** -23) * u.abs().mean(-1, keepdim=True) + 2.0 ** -21 * (u.abs() + s1.abs()))
    close(out["dx"], r64 * (u - s1), tol)

@pytest.mark.parametrize("D", [3, 5, 7, 24, 49, 60, 100, 131, 300, 513, 768, 771, 1000, 1600, 3001, 6000, 20011])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_constant_rows_have_their_value_as_mean(D, dtype):
    """Whole numbers whose sum is exact in fp32: the mean is the value and nothing is left of the row."""
    value = torch.arange(1.0, 51.0)
    x = value[:, None].expand(50, D).to(DT[dtype]).contiguous().cuda()
    b = torch.randn(D, device="cuda")
    y, mean, rstd = ttm.layer_norm_fwd(x, None, b)
    assert torch.equal(mean.cpu(), value)
    assert torch.equal(y, b.to(DT[dtype]).expand(50, D))


def test_a_row_of_2_to_the_30():
    """One row whose two sums take 2^31 words: the last columns count, and those of dw and db beyond 2^31."""
    D = 2 ** 30 + 3
    x = torch.ones(1, D, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -1                                   # n = x for mean 0 and rstd 1; sum x = 1
    y, mean, rstd = ttm.layer_norm_fwd(x)
    # a thread's 2^21 values have one sign, so its sums are exact; the mean is 1 / D, rstd off by 1e-5 / 2
    assert abs(float(mean)) < 2.0 ** -20 and abs(float(rstd) - 1) < 1e-5
    assert torch.equal(y, x)
    del y
    out = ttm.layer_norm_bwd(x, x, torch.zeros(1, device="cuda"), torch.ones(1, device="cuda"))
    assert bool((out["dw"] == 1).all()) and torch.equal(out["db"], x[0].float())
    assert float(out["dx"].abs().max()) < 2.0 ** -20   # x - 1 / D - x (1 - 3 2^-30), sums to 2^-24
