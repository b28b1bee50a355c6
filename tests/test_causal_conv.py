"""Short causal convolution, its gradient and its decode step against float64.

Tolerances, elementwise.  A sum of K products and a bias errs by at most e = (K + 1) 2^-24 of the sum of
sizes.  The logistic function s of x is off by at most q = (5 + 1.2 |x|) 2^-23 of itself (exponential:
2 + 1.2 |x| units at most in the fast form, a sum, a division of 2 units), SiLU by that share of itself and 1.1 e
more (its slope is at most 1.1), its slope by (q + 3 2^-23) (s + |x| s) + 0.5 e (the second derivative is at
most 0.5).  Sums of n terms in 32 bits err by at most n 2^-24 of the sum of sizes.  A bf16 result adds 2^-8 of itself."""
import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


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
    bad = ~((got - ref).abs() <= tol + HALF[dtype] * (ref.abs() + tol) + 1e-35)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


def make(N, T, C, K, dtype, bias=True, state=True, docs=False, pad=0, seed=0):
    r = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    wide = torch.randn((N, T, C + pad), generator=r).to(dt)
    dy = torch.randn((N, T, C + pad), generator=r).to(dt)
    w = torch.randn((C, K), generator=r)
    b = torch.randn((C,), generator=r) if bias else None
    s0 = torch.randn((N, K - 1, C), generator=r).to(dt) if state else None
    ds = torch.randn((N, K - 1, C), generator=r).to(dt)
    doc = (torch.rand((N, T), generator=r) < 0.2).cumsum(1).int() if docs else None
    return wide[..., :C], dy[..., :C], w, b, s0, ds, doc


def reference(x, dy, w, b, s0, ds, doc, silu):
    """Token by token: outputs, gradients, and the sums of sizes that the tolerances take."""
    N, T, C = x.shape
    K = w.shape[1]
    x, dy, w = x.double(), dy.double(), w.double()
    rows = torch.cat((torch.zeros(N, K - 1, C, dtype=torch.float64) if s0 is None else s0.double(), x), 1)
    ids = torch.zeros(N, T + K - 1, dtype=torch.int32)
    if doc is not None:
        ids[:, K - 1:] = doc
        ids[:, :K - 1] = doc[:, :1]
    pre = torch.zeros(N, T, C, dtype=torch.float64) + (0 if b is None else b.double())
    size = torch.zeros_like(pre) + (0 if b is None else b.double().abs())
    same = [(ids[:, i:i + T] == ids[:, K - 1:])[..., None] for i in range(K)]
    for i in range(K):
        tap = torch.where(same[i], rows[:, i:i + T], 0.0) * w[:, i]
        pre, size = pre + tap, size + tap.abs()
    e = (K + 1) * U * size
    s = torch.sigmoid(pre)
    q = (5 + 1.2 * pre.abs()) * 2 * U
    y, ty = (pre * s, (pre * s).abs() * q + 1.1 * e) if silu else (pre, e)
    slope = s * (1 + pre * (1 - s)) if silu else torch.ones_like(pre)
    ts = (q + 6 * U) * (s + pre.abs() * s) + 0.5 * e if silu else torch.zeros_like(pre)
    d, td = dy * slope, dy.abs() * ts
    drows, trows = torch.zeros_like(rows), torch.zeros_like(rows)
    dw, tw = torch.zeros_like(w), torch.zeros_like(w)
    n = N * T + 16
    for i in range(K):
        kept, tk = torch.where(same[i], d, 0.0), torch.where(same[i], td + (K + 2) * U * d.abs(), 0.0)
        drows[:, i:i + T] += kept * w[:, i]
        trows[:, i:i + T] += tk * w[:, i].abs()
        seen = torch.where(same[i], rows[:, i:i + T], 0.0)
        dw[:, i] = (d * seen).sum((0, 1))
        tw[:, i] = ((td + n * U * d.abs()) * seen.abs()).sum((0, 1))
    tail = (ids[:, T:] == ids[:, T + K - 2:T + K - 1])[..., None] if T else torch.ones(N, K - 1, 1, dtype=torch.bool)
    if K > 1:
        drows[:, T:] += torch.where(tail, ds.double(), 0.0)
        trows[:, T:] += 2 * U * (drows[:, T:].abs() + ds.double().abs())
    db, tb = d.sum((0, 1)), (td + n * U * d.abs()).sum((0, 1))
    return dict(y=(y, ty), state=torch.where(tail, rows[:, T:], 0.0), dx=(drows[:, K - 1:], trows[:, K - 1:]),
                ds0=(drows[:, :K - 1], trows[:, :K - 1]), dw=(dw, tw), db=(db, tb))


on = lambda t: None if t is None else t.cuda()  # noqa: E731


def check(N, T, C, K, dtype, bias=True, state=True, docs=False, pad=0, silu=True, seed=0):
    x, dy, w, b, s0, ds, doc = make(N, T, C, K, dtype, bias, state, docs, pad, seed)
    r = reference(x, dy, w, b, s0, ds, doc, silu)
    gx = on(torch.empty(N, T, C + pad, dtype=x.dtype))[..., :C].copy_(x)
    gd = on(torch.empty(N, T, C + pad, dtype=x.dtype))[..., :C].copy_(dy)
    y, out = ttm.causal_conv_fwd(gx, on(w), on(b), state0=on(s0), doc=on(doc), silu=silu)
    close(y, *r["y"], DT[dtype])
    assert torch.equal(out.cpu().double(), r["state"])
    call = lambda: ttm.causal_conv_bwd(gd, gx, on(w), on(b), state0=on(s0), doc=on(doc), silu=silu, dstate=on(ds))  # noqa: E731
    g = call()
    close(g["dx"], *r["dx"], DT[dtype])
    close(g["dw"], *r["dw"])
    if bias:
        close(g["db"], *r["db"])
    else:
        assert g["db"] is None
    if state:
        close(g["dstate0"], *r["ds0"], DT[dtype])
    else:
        assert g["dstate0"] is None
    again = call()
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,T,C", [(1, 1, 1), (1, 2, 8), (2, 3, 7), (1, 5, 64), (3, 17, 33), (2, 130, 12),
                                   (1, 700, 96), (5, 64, 4), (2, 257, 520), (700, 1, 16)])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8])
def test_sizes(N, T, C, K, dtype):
    check(N, T, C, K, dtype, docs=(T + K) % 2 == 1, seed=N + T + C + K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias,state,docs,silu", [(False, False, False, True), (True, False, True, True),
                                                  (False, True, True, False), (True, True, False, False)])
@pytest.mark.parametrize("pad", [0, 1, 2, 4, 8])
def test_options_and_alignments(dtype, bias, state, docs, silu, pad):
    check(2, 90, 48, 4, dtype, bias, state, docs, pad, silu, seed=pad)
    check(1, 41, 24, 7, dtype, bias, state, docs, pad, silu, seed=pad)


def test_long_rows_of_few_and_many_channels():
    check(1, 20000, 3, 4, "bf16")
    check(1, 9001, 40, 4, "f32", docs=True)
    check(2, 300, 2304, 4, "bf16", docs=True, pad=804)


def test_time_first_and_leading_dimensions():
    x, dy, w, b, s0, ds, _ = make(6, 50, 32, 4, "bf16")
    r = reference(x, dy, w, b, s0, ds, None, True)
    first = on(x.transpose(0, 1).contiguous()).transpose(0, 1)       # [T][N][C] in memory
    assert not first.is_contiguous()
    y, st = ttm.causal_conv_fwd(first, on(w), on(b), state0=on(s0))
    close(y, *r["y"], torch.bfloat16)
    g = ttm.causal_conv_bwd(on(dy.transpose(0, 1).contiguous()).transpose(0, 1), first, on(w), on(b), state0=on(s0), dstate=on(ds))
    close(g["dx"], *r["dx"], torch.bfloat16)
    y2, st2 = ttm.causal_conv_fwd(on(x).view(2, 3, 50, 32), on(w), on(b), state0=on(s0).view(2, 3, 3, 32))
    assert torch.equal(y2.view(6, 50, 32), y) and torch.equal(st2.view(6, 3, 32), st)
    same = on(x)[:1].expand(4, 50, 32)                               # one sequence read four times
    y3, _ = ttm.causal_conv_fwd(same.contiguous(), on(w), on(b))
    with pytest.raises(ttm.TTMError):
        ttm.causal_conv_fwd(same, on(w), on(b))
    assert torch.equal(y3[0], y3[3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 4, 6])
def test_steps_continue_a_pass(dtype, K):
    """A pass over a prefix, then steps of 1, 2, 1 and 7 tokens: the bits of one pass over everything."""
    x, _, w, b, s0, _, _ = make(3, 40, 24, K, dtype)
    x, w, b, s0 = on(x), on(w), on(b), on(s0)
    whole, last = ttm.causal_conv_fwd(x, w, b, state0=s0)
    y, state = ttm.causal_conv_fwd(x[:, :29], w, b, state0=s0)
    parts, at = [y], 29
    for n in (1, 2, 1, 7):
        parts.append(ttm.causal_conv_step(x[:, at:at + n], w, state, b))
        at += n
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, last)


def test_no_tokens():
    x, _, w, b, s0, ds, _ = make(2, 0, 8, 4, "bf16")
    y, state = ttm.causal_conv_fwd(on(x), on(w), on(b), state0=on(s0))
    assert y.shape == (2, 0, 8) and torch.equal(state.cpu(), s0)
    assert not ttm.causal_conv_fwd(on(x), on(w))[1].any()
    g = ttm.causal_conv_bwd(on(x), on(x), on(w), on(b), state0=on(s0), dstate=on(ds))
    assert torch.equal(g["dstate0"].cpu(), ds) and not g["dw"].any() and not g["db"].any()


def test_documents_are_independent():
    """A packed row gives the bits of its documents one by one, whatever the other documents hold."""
    x, dy, w, b, _, _, _ = make(1, 60, 16, 4, "f32")
    doc = torch.tensor([[0] * 1 + [1] * 2 + [7] * 30 + [2] * 27], dtype=torch.int32)
    x[0, 1:3] = float("nan")
    x[0, 32] = float("inf")
    y, state = ttm.causal_conv_fwd(on(x), on(w), on(b), doc=on(doc))
    g = ttm.causal_conv_bwd(on(dy), on(x), on(w), on(b), doc=on(doc))
    for lo, hi in ((0, 1), (3, 33), (33, 60)):
        part = on(x[:, lo:hi].contiguous())
        yp, sp = ttm.causal_conv_fwd(part, on(w), on(b))
        gp = ttm.causal_conv_bwd(on(dy[:, lo:hi].contiguous()), part, on(w), on(b))
        assert torch.equal(y[:, lo:hi].nan_to_num(7.0), yp.nan_to_num(7.0))
        assert torch.equal(g["dx"][:, lo:hi].nan_to_num(7.0), gp["dx"].nan_to_num(7.0))
    assert torch.equal(state, sp) and torch.isfinite(state).all()


def test_one_row_of_documents_for_every_sequence():
    x, dy, w, b, _, _, doc = (on(t) for t in make(3, 50, 24, 4, "bf16", docs=True))
    row = doc[:1].expand(3, 50)
    y, st = ttm.causal_conv_fwd(x, w, b, doc=row)
    want, wst = ttm.causal_conv_fwd(x, w, b, doc=row.contiguous())
    assert torch.equal(y, want) and torch.equal(st, wst)
    g, r = (ttm.causal_conv_bwd(dy, x, w, b, doc=d) for d in (row, row.contiguous()))
    assert torch.equal(g["dx"], r["dx"]) and torch.equal(g["dw"], r["dw"])


def test_offsets_past_32_bits():
    """2.3e9 values: the last tokens of a long row as short calls give them; as many sequences are refused (N C of 2^31
    and more)."""
    T, C = 140001, 16384
    r = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((1, T, C), generator=r, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((C, 4), generator=r, device="cuda")
    y, st = ttm.causal_conv_fwd(x, w)
    tail = x[:, -500:].contiguous()
    part, pst = ttm.causal_conv_fwd(tail[:, 3:], w, state0=tail[:, :3].contiguous())
    assert torch.equal(y[:, -497:], part) and torch.equal(st, pst)
    del y
    out = dict(dx=torch.empty_like(x))
    g = ttm.causal_conv_bwd(x, x, w, want_dw=False, out=out)
    gp = ttm.causal_conv_bwd(tail[:, 3:], tail[:, 3:], w, state0=tail[:, :3].contiguous(), want_dw=False)
    assert torch.equal(g["dx"][:, -497:], gp["dx"])
    many = x.view(T, 1, C)
    with pytest.raises(ttm.TTMError) as e:
        ttm.causal_conv_fwd(many, w)
    assert e.value.code == ttm.ERR_UNSUPPORTED
    y, _ = ttm.causal_conv_fwd(many[-131071:], w)
    assert torch.equal(y[-9:], ttm.causal_conv_fwd(many[-9:].contiguous(), w)[0])


def test_gradient_against_differences():
    """Central differences in float64 (step 1e-5, error about 1e-9) of <dy, y> + <ds, state>."""
    x, dy, w, b, s0, ds, doc = make(2, 6, 3, 3, "f32", docs=True, seed=5)

    def loss(x, w, b, s0):
        r = reference(x, dy, w, b, s0, ds, doc, True)
        return float((dy.double() * r["y"][0]).sum() + (ds.double() * r["state"]).sum())
    g = ttm.causal_conv_bwd(on(dy), on(x), on(w), on(b), state0=on(s0), doc=on(doc), dstate=on(ds))
    args = [t.double() for t in (x, w, b, s0)]
    for i, key in enumerate(("dx", "dw", "db", "dstate0")):
        for at in range(args[i].numel()):
            lo, hi = [a.clone() for a in args], [a.clone() for a in args]
            lo[i].view(-1)[at] -= 1e-5
            hi[i].view(-1)[at] += 1e-5
            want = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(float(g[key].reshape(-1)[at]) - want) < 2e-5 * (1 + abs(want)), (key, at)


def test_values_far_from_zero():
    """SiLU where its exponential overflows or vanishes."""
    x = torch.tensor([-1e30, -200.0, -90.0, -88.0, -20.0, 0.0, 20.0, 200.0, 1e30]).view(1, 9, 1)
    for dtype in ("f32", "bf16"):
        v = x.to(DT[dtype])
        one = torch.ones(1, 1)
        r = reference(v, torch.ones_like(v), one, None, None, torch.zeros(1, 0, 1), None, True)
        y, _ = ttm.causal_conv_fwd(on(v), on(one))
        g = ttm.causal_conv_bwd(on(torch.ones_like(v)), on(v), on(one))
        assert torch.isfinite(y).all() and torch.isfinite(g["dx"]).all()
        close(y, r["y"][0], r["y"][1] * (r["y"][0].abs() < 1e20) + 1e-32, DT[dtype])
        close(g["dx"], r["dx"][0].clamp(-1, 2), torch.full_like(r["dx"][0], 1e-5), DT[dtype])


def test_streams_graphs_and_given_outputs():
    x, dy, w, b, s0, ds, doc = (on(t) for t in make(2, 100, 64, 4, "bf16", docs=True))
    want, wst = ttm.causal_conv_fwd(x, w, b, state0=s0, doc=doc)
    wg = ttm.causal_conv_bwd(dy, x, w, b, state0=s0, doc=doc, dstate=ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, st = ttm.causal_conv_fwd(x, w, b, state0=s0, doc=doc, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(st, wst)
    y, st = torch.zeros_like(want), torch.zeros_like(wst)
    out = {k: torch.zeros_like(v) for k, v in wg.items()}
    state = s0.clone()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ttm.causal_conv_fwd(x, w, b, state0=s0, doc=doc, y=y, state=st)
            ttm.causal_conv_bwd(dy, x, w, b, state0=s0, doc=doc, dstate=ds, out=out)
            ys = ttm.causal_conv_step(x[:, :1], w, state, b)
    state.copy_(s0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(st, wst) and all(torch.equal(out[k], wg[k]) for k in wg)
    first = ys.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state[:, 1:], x[:, :1].expand(2, 2, 64)) and not torch.equal(first, ys)
    none = ttm.causal_conv_bwd(dy, x, w, b, state0=s0, doc=doc, dstate=ds, want_dw=False)
    assert none["dw"] is None and none["db"] is None and torch.equal(none["dx"], wg["dx"])


def test_refusals():
    x, w = torch.randn(2, 5, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    bad = [lambda: ttm.causal_conv_fwd(x[0, 0], w), lambda: ttm.causal_conv_fwd(x.cpu(), w),
           lambda: ttm.causal_conv_fwd(x, w[:7]), lambda: ttm.causal_conv_fwd(x, w.bfloat16()),
           lambda: ttm.causal_conv_fwd(x.transpose(1, 2), w), lambda: ttm.causal_conv_fwd(x, w, w[0]),
           lambda: ttm.causal_conv_fwd(x, w, state0=torch.zeros(2, 4, 8, device="cuda")),
           lambda: ttm.causal_conv_fwd(x, w, state0=torch.zeros(2, 3, 8, device="cuda", dtype=torch.bfloat16)),
           lambda: ttm.causal_conv_fwd(x, w, doc=torch.zeros(2, 5, device="cuda")),
           lambda: ttm.causal_conv_fwd(x, w, doc=torch.zeros(2, 4, device="cuda", dtype=torch.int32)),
           lambda: ttm.causal_conv_fwd(x, torch.randn(8, 9, device="cuda")),
           lambda: ttm.causal_conv_fwd(x, w, y=x), lambda: ttm.causal_conv_bwd(x[:, :4], x, w),
           lambda: ttm.causal_conv_bwd(x, x, w, out=dict(dx=x)),
           lambda: ttm.causal_conv_step(x[:, :0], w, torch.zeros(2, 3, 8, device="cuda")),
           lambda: ttm.causal_conv_step(x, w, torch.zeros(2, 2, 8, device="cuda"))]
    for call in bad:
        with pytest.raises(ttm.TTMError):
            call()
    with pytest.raises(TypeError):
        ttm.causal_conv_fwd(x.half(), w)
