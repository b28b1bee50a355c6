"""Cases of the training and decoding operators around the memory scan, each with its plain form.

  glr_fwd / glr_bwd / glr_step   gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per sequence and
                                 channel; its gradient; its form for a few tokens on a resident state
  ln_fwd / ln_bwd                layer norm over the last axis and its gradient
  ortho                          orthogonalised update by five quintic Newton-Schulz products

A case is a dict of sizes.  prepare() makes its inputs, run() makes one pass (the plain torch form in
32 bits, or the library's call where `own` is true), work() counts what a pass has to move and
compute, exact() is the definition in 64 bits.
"""
import functools
import math

import torch

own = False

EPS_LN = 1e-5
EPS_NS = 1e-7
# (a, b, c) of X <- a X + (b A + c A^2) X, A = X X^T, the same in each of the five steps
NS_COEFFS = ((3.4445, -4.7750, 2.0315),) * 5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

MOST_GLR = 16 * 131072 * 128         # elements of the longest recurrence listed
MOST_GLR_BWD = 96 * 8192 * 64
MOST_STEP = 4096 * 2048
MOST_LN = 131072 * 2048
MOST_NS = 5 * (4 * 2048 ** 2 * 8240 + 2 * 2048 ** 3)


def listed():
    return [
        # two packed prompts through a 768-wide layer (12 heads of 64): x and g are columns of one
        # projection, documents inside a row start from nothing (g = -inf)
        dict(name="glr fwd prompt", op="glr_fwd", N=2, T=777, D=768, dtype="bf16", gate="channel",
             h0=False, resets=True, pad=8),
        # the long-context shape: 16 heads of 128 channels, 131072 tokens, continued from a state
        dict(name="glr fwd long", op="glr_fwd", N=16, T=131072, D=128, dtype="bf16", gate="channel",
             h0=True, resets=False, pad=0),
        # the gradient at an odd size in 32 bits, one gate per token as the memory's momentum has it
        dict(name="glr bwd odd fp32", op="glr_bwd", N=3, T=1000, D=199, dtype="fp32", gate="token",
             h0=True, resets=True, pad=0),
        # the gradient of a training step: 8 rows of 12 heads, 8192 tokens, 64 channels
        dict(name="glr bwd train", op="glr_bwd", N=96, T=8192, D=64, dtype="bf16", gate="channel",
             h0=False, resets=False, pad=0),
        # one token for 64 rows of 16 heads: the smallest call, where latency counts
        dict(name="glr step decode", op="glr_step", N=1024, T=1, D=128, dtype="bf16", gate="channel",
             h0=True, resets=False, pad=0),
        # four tokens a call for a large decode batch of a 2048-wide layer, one gate per token
        dict(name="glr step batch", op="glr_step", N=1024, T=4, D=2048, dtype="bf16", gate="token",
             h0=True, resets=False, pad=8),
        # one token of 64 sequences before a 2048-wide layer
        dict(name="ln fwd decode", op="ln_fwd", N=64, D=2048, dtype="bf16", affine=True, pad=0),
        # the norm of every head's read-out: 8 x 12 x 8192 rows of 64
        dict(name="ln fwd heads", op="ln_fwd", N=786432, D=64, dtype="bf16", affine=True, pad=0),
        # a short ragged batch of a 768-wide layer in 32 bits, x a column slice of wider rows
        dict(name="ln bwd ragged fp32", op="ln_bwd", N=1537, D=768, dtype="fp32", affine=True, pad=3),
        # the gradient over the long-context batch of a 2048-wide layer
        dict(name="ln bwd long", op="ln_bwd", N=131072, D=2048, dtype="bf16", affine=True, pad=0),
        # the updates of every head's initial memory: 12 layers of 16 heads, 128 x 128
        dict(name="ortho heads", op="ortho", batch=192, m=128, n=128, dtype="fp32"),
        # the update of the input projection of a 2048-wide memory layer (4 D + 3 H columns)
        dict(name="ortho projection", op="ortho", batch=1, m=2048, n=8240, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("glr_fwd", "glr_bwd", "glr_step", "ln_fwd", "ln_bwd", "ortho"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op in ("glr_fwd", "glr_bwd"):
        most = (MOST_GLR if op == "glr_fwd" else MOST_GLR_BWD) // (2 if dtype == "fp32" else 1)
        T = _log(rng, 1, 131072)
        D = rng.choice((64, 128, 256, 768, 2048, _log(rng, 1, 2048), _log(rng, 1, 2048)))
        N = _log(rng, 1, max(1, min(4096, most // (T * D))))
        return dict(op=op, N=N, T=T, D=D, dtype=dtype, gate=rng.choice(("channel", "channel", "token")),
                    h0=rng.random() < 0.5, resets=rng.random() < 0.5, pad=rng.choice((0, 0, 8, 3)))
    if op == "glr_step":
        T, D = rng.choice((1, 1, 2, 3, 4, 7)), _log(rng, 16, 4096)
        N = _log(rng, 1, max(1, min(65536, MOST_STEP // (T * D))))
        return dict(op=op, N=N, T=T, D=D, dtype=dtype, gate=rng.choice(("channel", "token")), h0=True,
                    resets=False, pad=rng.choice((0, 8, 3)))
    if op in ("ln_fwd", "ln_bwd"):
        D = rng.choice((64, 128, 768, 2048, _log(rng, 2, 16384), _log(rng, 2, 16384)))
        N = _log(rng, 1, max(1, min(1 << 21, MOST_LN // (D * (2 if dtype == "fp32" else 1)))))
        return dict(op=op, N=N, D=D, dtype=dtype, affine=rng.random() < 0.8, pad=rng.choice((0, 0, 8, 3)))
    m, n = _log(rng, 8, 2048), _log(rng, 8, 8240)
    if rng.random() < 0.5:
        m, n = n, m
    r = min(m, n)
    batch = _log(rng, 1, max(1, min(1024, MOST_NS // (5 * (4 * r * m * n + 2 * r ** 3)), (1 << 26) // (m * n))))
    return dict(op=op, batch=batch, m=m, n=n, dtype=dtype)


# ------------------------------------------------------------------------------------- inputs

def _rows(gen, N, T, D, parts, pad, dtype):
    """`parts` tensors [N, T, D] of normal values: columns of one projection's rows when pad > 0."""
    if pad == 0:
        return [torch.randn((N, T, D), generator=gen, device="cuda", dtype=dtype) for _ in range(parts)]
    buf = torch.randn((N, T, parts * D + pad), generator=gen, device="cuda", dtype=dtype)
    return [buf[..., i * D:(i + 1) * D] for i in range(parts)]


def _glr_inputs(case, gen):
    N, T, D, dt = case["N"], case["T"], case["D"], DTYPES[case["dtype"]]
    if case["gate"] == "channel":
        x, g = _rows(gen, N, T, D, 2, case["pad"], dt)
    else:
        x, = _rows(gen, N, T, D, 1, case["pad"], dt)
        g = torch.randn((N, T), generator=gen, device="cuda")
    # retention 1 - alpha with alpha = 0.05 sigmoid(normal), as the memory's forgetting gate
    g.copy_(torch.log1p(-0.05 * torch.sigmoid(g.float())))
    if case["resets"]:
        at = torch.rand((N, T), generator=gen, device="cuda") < 1 / 256
        g.masked_fill_(at[..., None] if g.dim() == 3 else at, -math.inf)
    h0 = torch.randn((N, D), generator=gen, device="cuda") if case["h0"] else None
    return x, g, h0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = functools.partial(torch.randn, generator=gen, device="cuda")
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "glr_fwd":
        x, g, h0 = _glr_inputs(case, gen)
        return dict(op=op, x=x, g=g, h0=h0)
    if op == "glr_bwd":
        x, g, h0 = _glr_inputs(case, gen)
        h, h_last = _plain_glr_fwd(x, g, h0)
        return dict(op=op, g=g, h=h, h0=h0, dh=rand(h.shape, dtype=dt), dh_last=rand(h_last.shape))
    if op == "glr_step":
        x, g, state = _glr_inputs(case, gen)
        return dict(op=op, x=x, g=g, state=state)
    N, D = case.get("N"), case.get("D")
    if op == "ln_fwd" or op == "ln_bwd":
        x = rand((N, D + case["pad"]), dtype=dt)[:, :D]
        x.add_(0.5 * rand((D,), dtype=dt))
        w = 1 + 0.1 * rand((D,)) if case["affine"] else None
        b = 0.1 * rand((D,)) if case["affine"] else None
        if op == "ln_fwd":
            return dict(op=op, x=x, w=w, b=b)
        _, mean, rstd = _plain_ln_fwd(x, w, b)
        return dict(op=op, x=x, w=w, mean=mean, rstd=rstd, dy=rand((N, D), dtype=dt))
    # a momentum buffer: a few strong directions over noise
    m, n, r = case["m"], case["n"], min(8, case["m"], case["n"])
    G = rand((case["batch"], m, n))
    G.baddbmm_(rand((case["batch"], m, r)), rand((case["batch"], r, n)), alpha=2 / math.sqrt(r))
    return dict(op=op, G=G.to(dt))


# --------------------------------------------------------------------------------- plain forms

def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along axis 1 from zero: pairs of tokens joined, the scan of half the
    length, and the tokens between filled in."""
    T = x.shape[1]
    if T == 1:
        return x
    even = T // 2 * 2
    odd = _scan(a[:, 1:even:2] * a[:, 0:even:2], a[:, 1:even:2] * x[:, 0:even:2] + x[:, 1:even:2])
    h = torch.empty_like(x)
    h[:, 0] = x[:, 0]
    h[:, 1:even:2] = odd
    h[:, 2::2] = a[:, 2::2] * odd[:, :(T - 1) // 2] + x[:, 2::2]
    return h


def _decay(g):
    a = torch.exp(g.float())
    return a if g.dim() == 3 else a[..., None]


def _plain_glr_fwd(x, g, h0):
    a, h = _decay(g), x.to(torch.float32, copy=True, memory_format=torch.contiguous_format)
    if h0 is not None:
        h[:, 0] += a[:, 0] * h0
    h = _scan(a, h)
    return h.to(x.dtype), h[:, -1].clone()


def _plain_glr_bwd(g, h, h0, dh, dh_last):
    a, G = _decay(g), dh.float()
    G = G.clone() if G is dh else G
    G[:, -1] += dh_last
    # G_t = dh_t + a_{t+1} G_{t+1}: the same scan from the last token on
    G = _scan(torch.roll(a, -1, 1).flip(1), G.flip(1)).flip(1)
    c = a * G
    before = torch.zeros_like(h[:, :1], dtype=torch.float32) if h0 is None else h0[:, None]
    dg = c * torch.cat((before, h[:, :-1].float()), 1)
    dg = dg.to(g.dtype) if g.dim() == 3 else dg.sum(-1)
    return G.to(h.dtype), dg, c[:, 0].clone()


def _plain_ln_fwd(x, w, b):
    f = x.float()
    mean = f.mean(-1)
    d = f - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + EPS_LN)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w + b
    return y.to(x.dtype), mean, rstd


def _plain_ln_bwd(dy, x, w, mean, rstd):
    f = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    dw, db = (f * xhat).sum(0), f.sum(0)
    if w is not None:
        f = f * w
    dx = rstd[:, None] * (f - f.mean(-1, keepdim=True) - xhat * (f * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw, db


def _ns_step(X, coeffs):
    a, b, c = coeffs
    A = X @ X.mT
    return a * X + (b * A + c * (A @ A)) @ X


def _plain_ortho(G):
    X = G.float()
    X = X.mT if X.shape[1] > X.shape[2] else X
    X = X / torch.sqrt((X * X).sum((1, 2), keepdim=True)).clamp_min(EPS_NS)
    X = functools.reduce(_ns_step, NS_COEFFS, X)
    return (X.mT if G.shape[1] > G.shape[2] else X).to(torch.bfloat16).contiguous()


def _run_plain(s):
    op = s["op"]
    if op == "glr_fwd":
        h, h_last = _plain_glr_fwd(s["x"], s["g"], s["h0"])
        return dict(h=h, h_last=h_last)
    if op == "glr_bwd":
        dx, dg, dh0 = _plain_glr_bwd(s["g"], s["h"], s["h0"], s["dh"], s["dh_last"])
        return dict(dx=dx, dg=dg, dh0=dh0)
    if op == "glr_step":
        h, h_last = _plain_glr_fwd(s["x"], s["g"], s["state"])
        s["state"].copy_(h_last)
        return dict(h=h, state=s["state"])
    if op == "ln_fwd":
        y, mean, rstd = _plain_ln_fwd(s["x"], s["w"], s["b"])
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "ln_bwd":
        dx, dw, db = _plain_ln_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
        return dict(dx=dx, dw=dw, db=db)
    return dict(O=_plain_ortho(s["G"]))


def _run_own(s):
    import test_neural_memory_gb300 as ttm

    op = s["op"]
    if op == "glr_fwd":
        h, h_last = ttm.glr_fwd(s["x"], s["g"], h0=s["h0"])
        return dict(h=h, h_last=h_last)
    if op == "glr_bwd":
        return ttm.glr_bwd(s["g"], s["h"], s["dh"], h0=s["h0"], dh_last=s["dh_last"])
    if op == "glr_step":
        return dict(h=ttm.glr_step(s["x"], s["g"], s["state"]), state=s["state"])
    if op == "ln_fwd":
        y, mean, rstd = ttm.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS_LN)
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "ln_bwd":
        return ttm.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    return dict(O=ttm.orthogonalize(s["G"], coeffs=NS_COEFFS, eps=EPS_NS))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------- work, exactly

def work(case):
    op, es = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "ortho":
        r, b, mn = min(case["m"], case["n"]), case["batch"], case["m"] * case["n"]
        # per step A (its lower half), A^2 (its lower half) and the product with X
        return dict(bytes=b * mn * (es + 2), flops=b * 5 * (r * (r + 1) * (mn // r) + r * r * (r + 1) + 2 * r * mn))
    N, D = case["N"], case["D"]
    if op in ("ln_fwd", "ln_bwd"):
        vec = 8 * D if case["affine"] else 0
        if op == "ln_fwd":
            return dict(bytes=2 * N * D * es + 8 * N + vec, flops=8 * N * D)
        return dict(bytes=3 * N * D * es + 8 * N + vec // 2 + 8 * D, flops=13 * N * D)
    T = case["T"]
    gate = N * T * D * es if case["gate"] == "channel" else N * T * 4
    if op == "glr_bwd":
        return dict(bytes=3 * N * T * D * es + 2 * gate + (3 if case["h0"] else 2) * 4 * N * D, flops=5 * N * T * D)
    return dict(bytes=2 * N * T * D * es + gate + (2 if case["h0"] else 1) * 4 * N * D, flops=3 * N * T * D)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if op == "ortho":
        G = f64(s["G"])
        wide = G.shape[1] <= G.shape[2]
        X = G / torch.linalg.vector_norm(G, dim=(1, 2), keepdim=True).clamp_min(EPS_NS)
        for a, b, c in NS_COEFFS:
            # on the shorter side: X X^T X and (X X^T)^2 X
            gram = torch.matmul(X, X.transpose(1, 2)) if wide else torch.matmul(X.transpose(1, 2), X)
            X1 = torch.matmul(gram, X) if wide else torch.matmul(X, gram)
            X2 = torch.matmul(gram, X1) if wide else torch.matmul(X1, gram)
            X = a * X + b * X1 + c * X2
        return dict(O=X)
    if op == "ln_fwd":
        x = f64(s["x"])
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS_LN)
        y = torch.addcmul(-(mean * rstd)[:, None], x, rstd[:, None])
        return dict(y=y if s["w"] is None else torch.addcmul(f64(s["b"]), y, f64(s["w"])), mean=mean, rstd=rstd)
    if op == "ln_bwd":
        dy, x, rstd = f64(s["dy"]), f64(s["x"]), f64(s["rstd"])
        n = (x - f64(s["mean"])[:, None]).mul_(rstd[:, None])
        dw, db = torch.einsum("nd,nd->d", dy, n), torch.einsum("nd->d", dy)
        u = dy if s["w"] is None else dy * f64(s["w"])
        D = x.shape[1]
        dx = u - u.sum(1, keepdim=True) / D - n * (torch.einsum("nd,nd->n", u, n) / D)[:, None]
        return dict(dx=dx * rstd[:, None], dw=dw, db=db)
    keep = torch.exp(f64(s["g"]))
    keep = keep if keep.dim() == 3 else keep.unsqueeze(-1)
    T = keep.shape[1]
    if op == "glr_bwd":
        dx, h, dh = torch.empty_like(s["dh"], dtype=torch.float64), s["h"], s["dh"]
        token = s["g"].dim() == 2
        dg = torch.empty_like(s["g"], dtype=torch.float64)
        carry = f64(s["dh_last"])
        zero = torch.zeros_like(carry)
        for t in range(T - 1, -1, -1):
            dx[:, t] = carry + dh[:, t]
            carry = keep[:, t] * dx[:, t]
            before = h[:, t - 1] if t else (zero if s["h0"] is None else s["h0"])
            dg[:, t] = (carry * before).sum(-1) if token else carry * before
        return dict(dx=dx, dg=dg, dh0=carry)
    x = s["x"]
    start = s["h0"] if op == "glr_fwd" else s["state"]
    carry = torch.zeros_like(x[:, 0], dtype=torch.float64) if start is None else f64(start)
    h = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for t in range(T):
        carry = torch.addcmul(x[:, t].double(), keep[:, t], carry)
        h[:, t] = carry
    return dict(h=h, h_last=carry) if op == "glr_fwd" else dict(h=h, state=carry)
