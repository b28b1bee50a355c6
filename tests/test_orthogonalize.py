"""Orthogonalised update against the same steps in float64.

Tolerance.  The products take fp16 operands (11 bits) and add in fp32; X itself is kept to
fp32's accuracy.  How far that takes the result from float64 depends on the spectrum (the steps
multiply small singular values by up to 3.4 each), so the test rounds the operands of a float64
run the same way and allows twice what that moves the result, plus the rounding of the result to
bf16 (2^-8 of a value at most, under 2^-9 in the norm) and 2e-4 for fp32 sums."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def steps64(G, coeffs, eps=1e-7, rounded=False):
    half = (lambda t: (t * 1024).half().double() / 1024) if rounded else (lambda t: t)
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    X = X / X.flatten(1).norm(dim=1)[:, None, None].clamp_min(eps)
    for a, b, c in coeffs:
        Y = half(X)
        A = half(Y @ Y.mT)
        X = a * X + half(b * A + c * (A @ A)) @ Y
    return X.mT if tall else X


def matrices(batch, m, n, kind, seed=0):
    r = torch.Generator().manual_seed(seed)
    G = torch.randn((batch, m, n), generator=r)
    if kind == "low rank":
        G = 0.1 * G + torch.randn((batch, m, 2), generator=r) @ torch.randn((batch, 2, n), generator=r)
    if kind == "one column":
        G *= 1e-3
        G[..., 0] += torch.randn((batch, m), generator=r)
    return G


def check(G, coeffs, **kw):
    O = ttm.orthogonalize(G.cuda(), coeffs=coeffs, **kw)
    assert O.dtype == torch.bfloat16 and O.shape == G.shape
    flat = G.reshape(-1, *G.shape[-2:])
    ref = steps64(flat, coeffs, **kw)
    moved = (steps64(flat, coeffs, rounded=True, **kw) - ref).flatten(1).norm(dim=1)
    err = (O.double().cpu().reshape(ref.shape) - ref).flatten(1).norm(dim=1)
    size = ref.flatten(1).norm(dim=1)
    assert bool((err <= 2 * moved + (2.0 ** -9 + 2e-4) * size).all()), (err / size, moved / size)


@pytest.mark.parametrize("batch,m,n", [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 8, 8), (2, 33, 65),
                                       (5, 64, 64), (4, 64, 40), (3, 128, 128), (2, 127, 128),
                                       (2, 128, 100), (300, 16, 24), (1, 129, 129), (2, 200, 131),
                                       (1, 96, 700), (1, 700, 96), (2, 256, 256), (1, 257, 1031),
                                       (1, 768, 777), (3, 640, 300), (2, 40, 2000), (1, 1999, 37),
                                       (1, 130, 3001), (1, 1601, 9), (3, 1300, 70), (3, 128, 1024),
                                       (2, 5, 130), (2, 1023, 128), (90, 64, 385), (1, 66, 643),
                                       (40, 260, 500), (41, 500, 260)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "low rank"])
def test_against_float64(batch, m, n, dtype, kind):
    check(matrices(batch, m, n, kind, seed=m + n).to(DT[dtype]), ttm.train.NS_COEFFS)


@pytest.mark.parametrize("m,n", [(64, 64), (100, 300), (300, 200)])
@pytest.mark.parametrize("steps", [0, 1, 2, 3, 9])
def test_step_counts_and_other_coefficients(m, n, steps):
    """The cubically convergent quintic (15/8, -10/8, 3/8), another triple in every step."""
    coeffs = [(1.875 - 0.01 * i, -1.25 + 0.01 * i, 0.375) for i in range(steps)]
    check(matrices(2, m, n, "normal"), coeffs)


@pytest.mark.parametrize("m,n", [(128, 128), (200, 400)])
def test_one_strong_column_and_scale(m, n):
    """Entries over a range of 1e4, and the same matrix scaled by powers of two: equal bits."""
    G = matrices(2, m, n, "one column")
    check(G, ttm.train.NS_COEFFS)
    a = ttm.orthogonalize(G.cuda())
    for s in (2.0 ** -20, 2.0 ** 30):
        assert torch.equal(a, ttm.orthogonalize((G * s).cuda(), eps=1e-12))


@pytest.mark.parametrize("m,n", [(64, 128), (300, 500)])
def test_zero_and_tiny(m, n):
    G = torch.zeros(3, m, n)
    G[1] = matrices(1, m, n, "normal")[0]
    G[2] = 1e-12 * G[1]
    check(G, ttm.train.NS_COEFFS)                  # below eps the norm is not divided out
    assert not ttm.orthogonalize(G.cuda())[0].any()


@pytest.mark.parametrize("m,n", [(64, 64), (300, 200)])
def test_nan_stays_in_its_matrix(m, n):
    G = matrices(3, m, n, "normal")
    clean = ttm.orthogonalize(G.cuda())
    G[1, 3, 4] = float("nan")
    O = ttm.orthogonalize(G.cuda())
    assert bool(torch.isnan(O[1].float()).all())
    assert torch.equal(O[0], clean[0]) and torch.equal(O[2], clean[2])


def test_singular_values_come_near_one():
    G = matrices(2, 128, 384, "normal")
    s = torch.linalg.svdvals(ttm.orthogonalize(G.cuda()).float())
    assert float(s.min()) > 0.6 and float(s.max()) < 1.25
    # the convergent quintic reaches an orthogonal matrix to the accuracy of its operands
    O = ttm.orthogonalize(G.cuda(), coeffs=[(1.875, -1.25, 0.375)] * 16).double()
    eye = O @ O.mT - torch.eye(128, device="cuda", dtype=torch.float64)
    assert float(eye.abs().max()) < 1e-2


def test_stream_workspace_and_repeat():
    G = matrices(2, 300, 200, "normal").cuda()
    want = ttm.orthogonalize(G)
    n = ttm.lib().ttm_orthogonalize_workspace_size(2, 300, 200)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    got = ttm.orthogonalize(G, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert got is out and torch.equal(out, want)


def test_refusals():
    G = torch.randn(2, 20, 30, device="cuda")
    bad = [lambda: ttm.orthogonalize(G[0, 0]), lambda: ttm.orthogonalize(G[:, :, :8]),
           lambda: ttm.orthogonalize(G, out=torch.empty_like(G)), lambda: ttm.orthogonalize(G, eps=0.0),
           lambda: ttm.orthogonalize(G, coeffs=[(1.0, 2.0)]), lambda: ttm.orthogonalize(G.cpu()),
           lambda: ttm.orthogonalize(G, coeffs=[(1.0, 2.0, float("inf"))]),
           lambda: ttm.orthogonalize(torch.randn(200, 300, device="cuda"),
                                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for f in bad:
        with pytest.raises(ttm.TTMError) as e:
            f()
        assert e.value.code == ttm.ERR_INVALID_ARG
    with pytest.raises(ttm.TTMError) as e:
        ttm.orthogonalize(G, coeffs=[(1.0, 0.0, 0.0)] * 33)
    assert e.value.code == ttm.ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        ttm.orthogonalize(G.half())


@pytest.mark.parametrize("batch,m,n", [(1, 128, 129), (3, 129, 100), (153, 65, 300), (2, 90, 234), (400, 3, 131),
                                       (7, 1000, 128), (5, 1001, 77), (2, 5000, 64), (1, 60, 5003), (2, 4998, 33),
                                       (700, 11, 286), (310, 200, 16), (310, 201, 15), (1, 128, 20011),
                                       (1, 9973, 127), (160, 1027, 48), (1, 2, 1025), (1, 1, 3001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "low rank"])
def test_short_side_of_up_to_128(batch, m, n, dtype, kind):
    """Where the steps run on A alone: an operand, a sum of two fp16 values, errs by 2^-22 of itself and A by
    2^-20 of its norm; the default steps let that grow by 3.4445^5 = 485 at most, 4.7e-4 in all."""
    G = matrices(batch, m, n, kind, seed=m * n).to(DT[dtype])
    O = ttm.orthogonalize(G.cuda())
    ref = steps64(G, ttm.train.NS_COEFFS)
    err, size = (O.double().cpu() - ref).flatten(1).norm(dim=1), ref.flatten(1).norm(dim=1)
    # a cluster (64 x 1024 at most) or the products (other coefficients) keep the bound above
    moved = (steps64(G, ttm.train.NS_COEFFS, rounded=True) - ref).flatten(1).norm(dim=1)
    alone = min(m, n) > 64 or max(m, n) > 1024 or batch * ((max(m, n) + 127) // 128) > 304
    slack = 4.7e-4 * size if alone else 2 * moved
    assert bool((err <= slack + (2.0 ** -9 + 2e-4) * size).all()), float((err / size).max())
    assert torch.equal(O, ttm.orthogonalize(G.cuda()))


@pytest.mark.parametrize("m,n", [(100, 300), (70, 1500), (1500, 40)])
@pytest.mark.parametrize("steps", [1, 2, 4, 12])
def test_short_side_step_counts(m, n, steps):
    """Coefficients in turn; twelve steps let a rounding grow too far for A alone."""
    coeffs = [((1.875, -1.25, 0.375), ttm.train.NS_COEFFS[0], (1.5, -0.5, 0.0))[i % 3] for i in range(steps)]
    check(matrices(2, m, n, "normal"), coeffs)


def test_short_side_zero_tiny_nan_and_scale():
    for m, n in ((100, 300), (3000, 50)):
        G = torch.zeros(4, m, n)
        G[1:] = matrices(3, m, n, "one column")
        G[2] *= 1e-12
        check(G, ttm.train.NS_COEFFS)
        clean = ttm.orthogonalize(G.cuda())
        assert not clean[0].any()
        a = ttm.orthogonalize((G[1:2] * 2.0 ** 30).cuda(), eps=1e-12)
        assert torch.equal(a, ttm.orthogonalize((G[1:2] * 2.0 ** -20).cuda(), eps=1e-12))
        G[1, 3, 4] = float("nan")
        O = ttm.orthogonalize(G.cuda())
        assert bool(torch.isnan(O[1].float()).all())
        assert torch.equal(O[0], clean[0]) and torch.equal(O[2:], clean[2:])


def test_offsets_past_32_bits():
    """530 matrices of 64 x 65536, 2.2e9 elements: the last one counts."""
    G = torch.zeros(530, 64, 65536, dtype=torch.bfloat16, device="cuda")
    last = matrices(1, 64, 65536, "normal").bfloat16()
    G[-1] = last[0].cuda()
    O = ttm.orthogonalize(G)
    ref = steps64(last, ttm.train.NS_COEFFS)[0]
    err = float((O[-1].double().cpu() - ref).norm() / ref.norm())
    assert err < 2.0 ** -9 + 2e-4 + 4.7e-4 and not O[:-1].any()


@pytest.mark.parametrize("batch,m,n", [(4, 128, 128), (2, 700, 30), (3, 100, 900), (1, 2, 5000), (2, 300, 400)])
def test_captured_in_a_graph(batch, m, n):
    G = matrices(batch, m, n, "normal").cuda()
    out = torch.empty(G.shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, ttm.lib().ttm_orthogonalize_workspace_size(batch, m, n)), dtype=torch.uint8,
                     device="cuda")
    ttm.orthogonalize(G, out=out, workspace=ws)
    want = [out.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ttm.orthogonalize(G, out=out, workspace=ws)
        ttm.orthogonalize(G, out=out, workspace=ws)
    G.copy_(matrices(batch, m, n, "low rank", seed=3))
    want.append(ttm.orthogonalize(G))
    out.zero_()
    ws.fill_(255)
    graph.replay()
    assert torch.equal(out, want[1]) and not torch.equal(*want)


def spectrum(batch, m, n, kind, seed=0):
    """Matrices of few directions, whose small singular values the steps never take to one."""
    r = torch.Generator().manual_seed(seed)
    if kind == "rank 1" or kind == "rank 8":
        k = 1 if kind == "rank 1" else 8
        return torch.randn((batch, m, k), generator=r) @ torch.randn((batch, k, n), generator=r)
    if kind == "rank 8 and noise":
        noise = torch.randn((batch, m, n), generator=r)
        return 0.01 * noise + torch.randn((batch, m, 8), generator=r) @ torch.randn((batch, 8, n), generator=r)
    k = min(m, n)                                     # singular values from 1 down to 1e-6
    u = torch.linalg.qr(torch.randn((batch, m, k), generator=r, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn((batch, n, k), generator=r, dtype=torch.float64))[0]
    s = torch.logspace(0, -6, k, dtype=torch.float64) if k > 1 else torch.ones(1, dtype=torch.float64)
    return ((u * s) @ v.mT).float()


@pytest.mark.parametrize("batch,m,n", [(1, 300, 500), (1, 512, 512), (1, 768, 777), (1, 600, 300),
                                       (1, 100, 900)])
@pytest.mark.parametrize("kind", ["rank 1", "rank 8", "rank 8 and noise", "1 to 1e-6"])
def test_few_directions(batch, m, n, kind):
    """The bound of check(), which lets X be rounded to fp16 as an operand but not as a state: what
    is lost of a small singular value grows by 3.4 in every later step."""
    check(spectrum(batch, m, n, kind, seed=m + n), ttm.train.NS_COEFFS)


@pytest.mark.parametrize("batch,m,n", [(4, 16, 24), (3, 64, 64), (2, 64, 100), (3, 128, 128), (2, 100, 128),
                                       (1, 60, 700), (1, 700, 60), (2, 1000, 50), (2, 500, 200), (2, 130, 200)])
@pytest.mark.parametrize("kind", ["rank 1", "rank 8", "rank 8 and noise", "1 to 1e-6", "normal", "low rank"])
def test_few_directions_and_short_sides(batch, m, n, kind):
    """The same bound where B's diagonal is a large part of it although X is far from orthogonal."""
    G = (matrices if kind in ("normal", "low rank") else spectrum)(batch, m, n, kind, seed=m + n)
    check(G, ttm.train.NS_COEFFS)


def steps_in_11_bits(G, coeffs):
    """steps64, and the same with every operand rounded to 11 significant bits whatever its size."""
    def half(t):
        f, e = torch.frexp(t)
        return torch.ldexp(torch.round(torch.ldexp(f, torch.tensor(11))), e - 11)

    out = []
    for rounded in (lambda t: t, half):
        X = G.double()
        tall = X.shape[-2] > X.shape[-1]
        X = X.mT if tall else X
        X = X / X.flatten(1).norm(dim=1)[:, None, None]
        for a, b, c in coeffs:
            Y = rounded(X)
            A = rounded(Y @ Y.mT)
            X = a * X + rounded(b * A + c * (A @ A)) @ Y
        out.append(X.mT if tall else X)
    return out


@pytest.mark.parametrize("m,n", [(2, 40), (64, 64), (128, 100), (60, 700), (100, 300), (900, 40), (300, 200)])
@pytest.mark.parametrize("coeffs", [[(1.0, -200.0, 0.0)], [(0.0, 0.0, 3e4)], [(0.0, 1e-7, 0.0)],
                                    [(40.0, 0.0, 0.0), (0.01, 0.0, 0.0)], [(100.0, 0.0, 0.0), (1.0, -1e-4, 3e-9)],
                                    [(1e6, 0.0, 0.0), (1e-6, 1e-18, 0.0)], [(1e-3, 0.0, 0.0)] * 3,
                                    [(1e-4, 0.0, 0.0), (0.0, 1e8, 0.0)]])
@pytest.mark.parametrize("kind", ["normal", "rank 1"])
def test_coefficients_of_any_size(m, n, coeffs, kind):
    """Finite coefficients whose polynomials are finite: the operands' scales follow them.  The bound is
    check()'s, with operands of 11 bits and no limit to their exponent."""
    G = matrices(2, m, n, "normal", seed=3) if kind == "normal" else spectrum(2, m, n, kind, seed=3)
    O = ttm.orthogonalize(G.cuda(), coeffs=coeffs).double().cpu()
    ref, rough = steps_in_11_bits(G, coeffs)
    err, moved, size = ((t - ref).flatten(1).norm(dim=1) for t in (O, rough, 0 * ref))
    assert bool((err <= 2 * moved + (2.0 ** -9 + 2e-4) * size).all()), (err / size, moved / size)


@pytest.mark.parametrize("m,n", [(64, 64), (40, 700), (100, 900), (300, 200)])
@pytest.mark.parametrize("eps", [1e-20, 1e-30, 1e-38])
def test_zero_with_a_tiny_eps(m, n, eps):
    G = torch.zeros(2, m, n)
    G[1] = matrices(1, m, n, "normal")[0]
    O = ttm.orthogonalize(G.cuda(), eps=eps)
    assert not O[0].any()
    assert torch.equal(O[1], ttm.orthogonalize(G.cuda())[1])


@pytest.mark.parametrize("batch,m,n", [(12, 100, 256), (12, 100, 900), (12, 128, 2000), (12, 50, 3000), (12, 2000, 128),
                                       (12, 900, 100), (4, 3000, 50), (5, 90, 390), (12, 17, 1300)])
@pytest.mark.parametrize("kind", ["rank 1", "rank 8", "rank 8 and noise", "1 to 1e-6", "one column"])
def test_few_directions_on_a_alone(batch, m, n, kind):
    """What the interface states: 3e-3 of the norm.  Its parts: 1.66e-3 for rounding to bf16; and sums that the
    tensor cores cut off at 24 bits, a few in a row, times the 485 that Q is on what X has nothing of."""
    G = (matrices if kind == "one column" else spectrum)(batch, m, n, kind, seed=5)
    ref = steps64(G, ttm.train.NS_COEFFS)
    err = (ttm.orthogonalize(G.cuda()).double().cpu() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert bool((err <= 3e-3).all()), err
