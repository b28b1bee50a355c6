"""Cases of the operators that complete a residual block around the memory scan, each with its plain form.

  conv_fwd / conv_bwd / conv_step   short causal depthwise convolution with SiLU; its gradient; its form for
                                    a few tokens on a resident state
  ffn_fwd / ffn_bwd                 gated feed-forward block act(x W_g) * (x W_u) W_o and its gradient
  adamw                             AdamW step over many tensors, moments in 32 bits or in 8

A case is a dict of plain values.  prepare() makes its inputs, run() makes one pass (the plain torch form in
32 bits, or the library's call where `own` is true), work() counts what a pass has to move and compute,
exact() is the definition in 64 bits.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 256                           # values of a moment that share a scale, and a tensor's start is a multiple of
BETAS, EPS, LR, DECAY = (0.9, 0.95), 1e-8, 3e-4, 0.1

MOST_CONV = 131072 * 6144             # values of the longest convolution listed
MOST_CONV_BWD = 8 * 8192 * 2304
MOST_STEP = 4096 * 6144
MOST_FFN = 32768 * 2048 * 5504        # rows x width x hidden width, forward
MOST_ADAMW = 1 << 27                  # values of a drawn optimiser step


def listed():
    return [
        # two packed prompts through the q, k and v columns of a 768-wide layer's projection (12 heads of 64;
        # rows of 4 x 768 + 36 values); documents start inside the rows
        dict(name="conv fwd prompt", op="conv_fwd", N=2, T=777, C=2304, K=4, dtype="bf16", bias=False, silu=True,
             state=False, docs=True, pad=804),
        # the long-context shape: q, k and v of 16 heads of 128, continued from a prefix
        dict(name="conv fwd long", op="conv_fwd", N=1, T=131072, C=6144, K=4, dtype="bf16", bias=False, silu=True,
             state=True, docs=False, pad=2096),
        # the gradient at odd sizes in 32 bits, three taps with a bias
        dict(name="conv bwd odd fp32", op="conv_bwd", N=3, T=1000, C=199, K=3, dtype="fp32", bias=True, silu=True,
             state=True, docs=True, pad=0),
        # the gradient of a training step: 8 rows of 8192 tokens, q, k and v of 12 heads of 64
        dict(name="conv bwd train", op="conv_bwd", N=8, T=8192, C=2304, K=4, dtype="bf16", bias=False, silu=True,
             state=False, docs=False, pad=804),
        # one token of 64 sequences of a 2048-wide layer: the smallest call, where latency counts
        dict(name="conv step decode", op="conv_step", N=64, T=1, C=6144, K=4, dtype="bf16", bias=False, silu=True,
             state=True, docs=False, pad=0),
        # one token of 16 sequences through the block of a 2048-wide layer: the weights are what is read
        dict(name="ffn fwd decode", op="ffn_fwd", N=16, D=2048, F=5504, act="silu", residual=True, save=False, pad=0),
        # the forward pass of a training step over 32768 tokens, g and u kept for the gradient
        dict(name="ffn fwd long", op="ffn_fwd", N=32768, D=2048, F=5504, act="silu", residual=True, save=True, pad=0),
        # the gradient of a short ragged batch of a 768-wide layer with GELU
        dict(name="ffn bwd ragged", op="ffn_bwd", N=1537, D=768, F=2056, act="gelu", residual=False, save=True, pad=8),
        # the gradient of a training step over 16384 tokens
        dict(name="ffn bwd train", op="ffn_bwd", N=16384, D=2048, F=5504, act="silu", residual=False, save=True, pad=0),
        # the norms, biases and taps of 12 layers, whose matrices take another update: many short tensors
        dict(name="adamw vectors", op="adamw", layers=12, width=768, matrices=False, bits=32, param="fp32",
             grad="fp32", copies=False, clip=True),
        # all of 12 layers of width 768: fp32 weights with the bf16 copies that the kernels read, bf16 gradients
        dict(name="adamw layers", op="adamw", layers=12, width=768, matrices=True, bits=32, param="fp32",
             grad="bf16", copies=True, clip=True),
        # four layers of width 2048 with the moments in 8 bits
        dict(name="adamw 8 bits", op="adamw", layers=4, width=2048, matrices=True, bits=8, param="fp32",
             grad="bf16", copies=True, clip=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("conv_fwd", "conv_bwd", "conv_step", "ffn_fwd", "ffn_bwd", "adamw"))
    if op.startswith("conv"):
        dtype = rng.choice(("bf16", "bf16", "fp32"))
        most = (MOST_CONV if op == "conv_fwd" else MOST_CONV_BWD) // (2 if dtype == "fp32" else 1)
        C = rng.choice((768, 2304, 6144, _log(rng, 1, 8192), _log(rng, 1, 8192)))
        if op == "conv_step":
            T = rng.choice((1, 1, 2, 5))
            N = _log(rng, 1, max(1, min(4096, MOST_STEP // (T * C))))
            docs = False
        else:
            T = _log(rng, 1, 131072)
            N = _log(rng, 1, max(1, min(2048, most // (T * C))))
            docs = rng.random() < 0.4
        return dict(op=op, N=N, T=T, C=C, K=rng.choice((4, 4, 3, 2, 7, 1)), dtype=dtype, bias=rng.random() < 0.5,
                    silu=rng.random() < 0.8, state=op == "conv_step" or rng.random() < 0.5, docs=docs,
                    pad=rng.choice((0, 0, 8, 3)))
    if op in ("ffn_fwd", "ffn_bwd"):
        D = rng.choice((512, 768, 2048, 8 * _log(rng, 8, 512)))
        F = rng.choice((2048, 5504, 8 * _log(rng, 8, 1024)))
        N = _log(rng, 1, min(65536, MOST_FFN // (D * F * (1 if op == "ffn_fwd" else 2))))
        return dict(op=op, N=N, D=D, F=F, act=rng.choice(("silu", "silu", "gelu")), residual=op == "ffn_fwd" and rng.random() < 0.5,
                    save=op == "ffn_bwd" or rng.random() < 0.5, pad=rng.choice((0, 0, 8)))
    param = rng.choice(("fp32", "fp32", "bf16"))
    largest = _log(rng, 8, 1 << 24)
    return dict(op=op, tensors=_log(rng, 1, max(1, min(300, MOST_ADAMW // largest))), largest=largest,
                mix=rng.randrange(1 << 30), bits=rng.choice((8, 32)), param=param, grad=rng.choice(("fp32", "bf16")),
                copies=param == "fp32" and rng.random() < 0.5, clip=rng.random() < 0.5)


def _sizes(case):
    """Values of each tensor of an optimiser step."""
    if "width" not in case:
        rng = random.Random(case["mix"])
        return [_log(rng, 1, case["largest"]) for _ in range(case["tensors"])]
    D, H = case["width"], case["width"] // (64 if case["width"] == 768 else 128)
    F = 2048 if D == 768 else 5504
    # two norms with their biases, the head norm, the taps and their bias, the gates' bias
    vectors = [D, D, D, D, D // H, 3 * D * 4, 3 * D, 3 * H]
    matrices = [D * (4 * D + 3 * H), D * D, 2 * D * F, F * D]
    return (vectors + matrices if case["matrices"] else vectors) * case["layers"]


def _ends(sizes, unit):
    """Where each tensor starts in a flat buffer of tensors of whole units, and the buffer's length."""
    at = [0]
    at.extend(at[-1] + (n + unit - 1) // unit * unit for n in sizes)
    return at[:-1], at[-1]


# ------------------------------------------------------------------------------------- inputs

def _columns(rand, N, T, D, pad, dtype):
    """[N, T, D] of normal values: columns of wider rows when pad > 0."""
    return rand((N, T, D + pad), dtype=dtype)[..., pad // 2 // 8 * 8:][..., :D]


def _prepare_conv(case, gen, rand):
    N, T, C, K, dt = case["N"], case["T"], case["C"], case["K"], DTYPES[case["dtype"]]
    x = _columns(rand, N, T, C, case["pad"], dt)
    w = rand((C, K)) / math.sqrt(K)
    b = 0.1 * rand((C,)) if case["bias"] else None
    state = rand((N, K - 1, C), dtype=dt) if case["state"] else None
    doc = None
    if case["docs"]:
        at = torch.rand((N, T), generator=gen, device="cuda") < 1 / 128
        doc = at.cumsum(1).to(torch.int32)
    s = dict(op=case["op"], x=x, w=w, b=b, state=state, doc=doc, silu=case["silu"])
    if case["op"] == "conv_bwd":
        s["dy"] = rand((N, T, C), dtype=dt)
        s["dstate"] = rand((N, K - 1, C), dtype=dt) if case["state"] else None
    return s


def _prepare_ffn(case, rand):
    N, D, F, bf = case["N"], case["D"], case["F"], torch.bfloat16
    x = _columns(rand, 1, N, D, case["pad"], bf)[0]
    W_in = (rand((D, 2 * F)) / math.sqrt(D)).to(bf)
    W_out = (rand((F, D)) / math.sqrt(F)).to(bf)
    s = dict(op=case["op"], x=x, W_in=W_in, W_out=W_out, act=case["act"], save=case["save"],
             residual=rand((N, D), dtype=bf) if case["residual"] else None)
    if case["op"] == "ffn_bwd":
        s["gu"] = (x.float() @ W_in.float()).to(bf)
        s["dy"] = rand((N, D), dtype=bf)
    return s


def _coded(values):
    """e4m3 values and a power of two for each block of BLOCK, the smallest that leaves none over 448."""
    blocks = values.view(-1, BLOCK)
    scale = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax(1).clamp_min(1e-30) / 448)))
    return (blocks / scale[:, None]).to(torch.float8_e4m3fn).view(-1), scale


def _prepare_adamw(case, gen, rand):
    sizes, dt = _sizes(case), DTYPES[case["param"]]
    packed, total = _ends(sizes, 1)
    first, held = _ends(sizes, BLOCK)
    flat = (0.05 * rand((total,))).to(dt)
    copy = flat.to(torch.bfloat16) if case["copies"] else None
    inside = torch.zeros(held, device="cuda")
    spread = torch.exp(rand((total,)))                 # gradients of several sizes in every tensor
    m, v, grads = torch.zeros(held, device="cuda"), torch.zeros(held, device="cuda"), []
    for n, a, f in zip(sizes, packed, first):
        inside[f:f + n] = 1e-3 * spread[a:a + n]
        grads.append((1e-3 * spread[a:a + n] * rand((n,))).to(DTYPES[case["grad"]]))
    m.copy_(0.3 * inside * rand((held,)))
    v.copy_((inside * (0.5 + torch.rand(held, generator=gen, device="cuda"))) ** 2)
    step = torch.tensor([100, 0], dtype=torch.int32, device="cuda")
    if case["bits"] == 8:
        (m, m_scale), (r, r_scale) = _coded(m), _coded(v.sqrt())
        state = dict(m=m, v=r, m_scale=m_scale, v_scale=r_scale, step=step)
    else:
        state = dict(m=m, v=v, step=step)
    cut = lambda t: [t[a:a + n] for n, a in zip(sizes, packed)]  # noqa: E731
    return dict(op="adamw", flat=flat, params=cut(flat), grads=grads, state=state, copy=copy,
                copies=None if copy is None else cut(copy), first=first,
                scale=torch.tensor(0.7, device="cuda") if case["clip"] else None)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = functools.partial(torch.randn, generator=gen, device="cuda")
    if case["op"].startswith("conv"):
        return _prepare_conv(case, gen, rand)
    if case["op"].startswith("ffn"):
        return _prepare_ffn(case, rand)
    return _prepare_adamw(case, gen, rand)


# --------------------------------------------------------------------------------- plain forms

def _ids(doc, before):
    """Document of every row of [state, x]: the state is of the first token's."""
    return torch.cat((doc[:, :1].expand(-1, before), doc), 1)


def _taps(x, state, doc, K):
    """[state, x], and which of its rows t + i reach token t."""
    N, T, C = x.shape
    rows = torch.cat((x.new_zeros((N, K - 1, C)) if state is None else state, x), 1)
    if doc is None:
        return rows, [None] * K
    ids = _ids(doc, K - 1)
    return rows, [(ids[:, i:i + T] == doc)[..., None] for i in range(K)]


def _kept(rows, mask):
    return rows.float() if mask is None else rows.float() * mask


def _conv_pre(rows, masks, w, b, T):
    pre = functools.reduce(lambda acc, i: acc + w[:, i] * _kept(rows[:, i:i + T], masks[i]), range(1, w.shape[1]),
                           w[:, 0] * _kept(rows[:, :T], masks[0]))
    return pre if b is None else pre + b


def _last_rows(rows, doc, K):
    """The last K - 1 rows of [state, x], zero where they are of another document than the last token."""
    last = rows[:, rows.shape[1] - (K - 1):]
    if doc is None:
        return last.clone()
    ids = _ids(doc, K - 1)
    return last * (ids[:, ids.shape[1] - (K - 1):] == doc[:, -1:])[..., None]


def _plain_conv_fwd(x, w, b, state, doc, silu):
    K, T = w.shape[1], x.shape[1]
    rows, masks = _taps(x, state, doc, K)
    pre = _conv_pre(rows, masks, w, b, T)
    y = pre / (1 + torch.exp(-pre)) if silu else pre
    return y.to(x.dtype), _last_rows(rows, doc, K)


def _plain_conv_bwd(dy, x, w, b, state, doc, silu, dstate):
    K, T = w.shape[1], x.shape[1]
    rows, masks = _taps(x, state, doc, K)
    d = dy.float()
    if silu:
        pre = _conv_pre(rows, masks, w, b, T)
        s = 1 / (1 + torch.exp(-pre))
        d = d * s * (1 + pre * (1 - s))
    drows = torch.zeros(rows.shape, device=x.device)
    dw = [(d * _kept(rows[:, i:i + T], masks[i])).sum((0, 1)) for i in range(K)]
    [drows[:, i:i + T].add_(_kept(w[:, i] * d, masks[i])) for i in range(K)]
    if dstate is not None and K > 1:
        keep = 1 if doc is None else (_ids(doc, K - 1)[:, T:] == doc[:, -1:])[..., None]
        drows[:, T:] += dstate.float() * keep
    return dict(dx=drows[:, K - 1:].to(x.dtype), dw=torch.stack(dw, 1), db=None if b is None else d.sum((0, 1)),
                dstate0=None if state is None else drows[:, :K - 1].to(x.dtype))


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))


def _act_slope(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g / math.sqrt(2))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _plain_ffn_fwd(x, W_in, W_out, act, residual):
    F = W_out.shape[0]
    gu = x.float() @ W_in.float()
    y = (_act(gu[:, :F], act) * gu[:, F:]) @ W_out.float()
    return (y if residual is None else y + residual).to(x.dtype), gu.to(x.dtype)


def _plain_ffn_bwd(dy, x, gu, W_in, W_out, act):
    F = W_out.shape[0]
    g, u, dy = gu[:, :F].float(), gu[:, F:].float(), dy.float()
    a = _act(g, act)
    dW_out = (a * u).T @ dy
    dh = dy @ W_out.float().T
    dgu = torch.cat((dh * u * _act_slope(g, act), dh * a), 1)
    return dict(dx=(dgu @ W_in.float().T).to(x.dtype), dW_in=(x.float().T @ dgu).to(x.dtype), dW_out=dW_out.to(x.dtype))


def _dither(first, n, step):
    """Two fractions in [0, 1) for each of the values first .. first + n - 1: a 32-bit integer hash of the value's
    place and the step, cut in two."""
    at = first + torch.arange(n, device=step.device)
    h = ((at & 0xffffffff) + step * 0x9e3779b9 + (at >> 32) * 0x85ebca6b) & 0xffffffff
    h = h ^ (h >> 16)
    h = (h * 0x7feb352d) & 0xffffffff
    h = h ^ (h >> 15)
    h = (h * 0x846ca68b) & 0xffffffff
    h = h ^ (h >> 16)
    return (h & 0xffff).float() / 65536, (h >> 16).float() / 65536


def _binade(t):
    """Exponent of a positive 32-bit value."""
    return (t.view(torch.int32) >> 23) - 127


def _power(e):
    return ((e + 127) << 23).view(torch.float32)


def _to_8_bits(t, frac):
    """The values in e4m3 times a power of two per block, rounded up where frac exceeds the step's missing part."""
    blocks = torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).view(-1, BLOCK)
    frac = torch.nn.functional.pad(frac, (0, -t.numel() % BLOCK)).view(-1, BLOCK)
    most = blocks.abs().amax(1)
    e = (_binade(most) - 8 + ((most.view(torch.int32) & 0x7fffff) > 0x600000)).clamp_min(-126)
    y = blocks.abs() * _power(-e)[:, None]
    b = _binade(y).clamp_min(-6)
    q = torch.floor(y * _power(3 - b) + frac) * _power(b - 3)
    return torch.copysign(q, blocks).view(-1)[:t.numel()].to(torch.float8_e4m3fn), _power(e)


def _decoded(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw_one(p, g, first, s, bias, copy):
    st, n = s["state"], p.numel()
    own_blocks = slice(first // BLOCK, (first + n + BLOCK - 1) // BLOCK)
    part = slice(first, first + n)
    if "m_scale" in st:
        whole = slice(first, own_blocks.stop * BLOCK)
        m = _decoded(st["m"][whole], st["m_scale"][own_blocks])[:n]
        r = _decoded(st["v"][whole], st["v_scale"][own_blocks])[:n]
        v = r * r
    else:
        m, v = st["m"][part], st["v"][part]
    g = g.float() if s["scale"] is None else g.float() * s["scale"]
    m = m * BETAS[0] + g * (1 - BETAS[0])
    v = v * BETAS[1] + g * g * (1 - BETAS[1])
    new = p.float() * (1 - LR * DECAY) - LR * (m / bias[0]) / (torch.sqrt(v / bias[1]) + EPS)
    p.copy_(new)
    if copy is not None:
        copy.copy_(new)
    if "m_scale" in st:
        up_m, up_r = _dither(first, n, st["step"][0].long() + 1)
        st["m"][part], st["m_scale"][own_blocks] = _to_8_bits(m, up_m)
        st["v"][part], st["v_scale"][own_blocks] = _to_8_bits(torch.sqrt(v), up_r)
    else:
        st["m"][part], st["v"][part] = m, v


def _plain_adamw(s):
    n = s["state"]["step"][0].double() + 1
    bias = [(1 - b ** n).float() for b in BETAS]
    copies = s["copies"] or [None] * len(s["params"])
    [_adamw_one(p, g, f, s, bias, c) for p, g, f, c in zip(s["params"], s["grads"], s["first"], copies)]
    s["state"]["step"][0] += 1
    return _adamw_outputs(s, _plain_moments(s["state"]))


def _plain_moments(st):
    if "m_scale" not in st:
        return st["m"], st["v"]
    r = _decoded(st["v"], st["v_scale"])
    return _decoded(st["m"], st["m_scale"]), r * r


def _adamw_outputs(s, moments):
    return dict(params=s["flat"], copies=s["copy"], m=moments[0], v=moments[1], step=s["state"]["step"])


def _run_plain(s):
    op = s["op"]
    if op == "conv_fwd":
        y, state = _plain_conv_fwd(s["x"], s["w"], s["b"], s["state"], s["doc"], s["silu"])
        return dict(y=y, state=state)
    if op == "conv_bwd":
        return _plain_conv_bwd(s["dy"], s["x"], s["w"], s["b"], s["state"], s["doc"], s["silu"], s["dstate"])
    if op == "conv_step":
        y, state = _plain_conv_fwd(s["x"], s["w"], s["b"], s["state"], None, s["silu"])
        s["state"].copy_(state)
        return dict(y=y, state=s["state"])
    if op == "ffn_fwd":
        y, gu = _plain_ffn_fwd(s["x"], s["W_in"], s["W_out"], s["act"], s["residual"])
        return dict(y=y, gu=gu if s["save"] else None)
    if op == "ffn_bwd":
        return _plain_ffn_bwd(s["dy"], s["x"], s["gu"], s["W_in"], s["W_out"], s["act"])
    return _plain_adamw(s)


def _run_own(s):
    import test_neural_memory_gb300 as ttm

    op = s["op"]
    if op == "conv_fwd":
        y, state = ttm.causal_conv_fwd(s["x"], s["w"], s["b"], state0=s["state"], doc=s["doc"], silu=s["silu"])
        return dict(y=y, state=state)
    if op == "conv_bwd":
        return ttm.causal_conv_bwd(s["dy"], s["x"], s["w"], s["b"], state0=s["state"], doc=s["doc"], silu=s["silu"],
                                   dstate=s["dstate"])
    if op == "conv_step":
        return dict(y=ttm.causal_conv_step(s["x"], s["w"], s["state"], s["b"], silu=s["silu"]), state=s["state"])
    if op == "ffn_fwd":
        y, gu = ttm.gated_ffn_fwd(s["x"], s["W_in"], s["W_out"], act=s["act"], residual=s["residual"], want_gu=s["save"])
        return dict(y=y, gu=gu)
    if op == "ffn_bwd":
        return ttm.gated_ffn_bwd(s["dy"], s["x"], s["gu"], s["W_in"], s["W_out"], act=s["act"])
    ttm.adamw_step(s["params"], s["grads"], s["state"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                   grad_scale=s["scale"], copies=s["copies"])
    return _adamw_outputs(s, ttm.adamw_moments(s["state"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------- work, exactly

def work(case):
    op = case["op"]
    if op.startswith("conv"):
        N, T, C, K = case["N"], case["T"], case["C"], case["K"]
        es = 4 if case["dtype"] == "fp32" else 2
        states = (2 if case["state"] else 1) * N * (K - 1) * C * es
        small = 4 * C * (K + (1 if case["bias"] else 0)) + (4 * N * T if case["docs"] else 0)
        if op == "conv_bwd":
            return dict(bytes=3 * N * T * C * es + (3 if case["state"] else 0) * N * (K - 1) * C * es + small
                        + 4 * C * (K + (1 if case["bias"] else 0)), flops=N * T * C * (6 * K + 10))
        return dict(bytes=2 * N * T * C * es + states + small, flops=N * T * C * (2 * K + 5))
    if op.startswith("ffn"):
        N, D, F = case["N"], case["D"], case["F"]
        weights = 2 * 3 * D * F
        if op == "ffn_fwd":
            return dict(bytes=weights + 2 * N * D * (3 if case["residual"] else 2) + (4 * N * F if case["save"] else 0),
                        flops=6 * N * D * F)
        return dict(bytes=2 * weights + 2 * N * D * 3 + 4 * N * F, flops=12 * N * D * F)
    sizes = _sizes(case)
    n, held = sum(sizes), _ends(sizes, BLOCK)[1]
    each = 2 * (4 if case["param"] == "fp32" else 2) + (4 if case["grad"] == "fp32" else 2) + (2 if case["copies"] else 0)
    # moments read and written; those in 8 bits also leave as values
    moments = 16 * n if case["bits"] == 32 else 4 * n + 16 * held // BLOCK + 8 * held
    return dict(bytes=each * n + moments, flops=14 * n)


def _exact_conv(s):
    x, w = s["x"].double(), s["w"].double()
    N, T, C = x.shape
    K = w.shape[1]
    state = x.new_zeros((N, K - 1, C)) if s["state"] is None else s["state"].double()
    rows = torch.cat((state, x), 1)
    place = torch.arange(T, device=x.device)
    same = torch.ones((N, T, K), dtype=torch.bool, device=x.device)
    if s["doc"] is not None:
        source = (place[:, None] + torch.arange(K, device=x.device) - (K - 1)).clamp_min(0)
        same = s["doc"][:, source] == s["doc"][:, :, None]
    return x, w, rows, same


def _exact_tail(s, rows, K):
    T = s["x"].shape[1]
    keep = torch.ones((rows.shape[0], K - 1), dtype=torch.bool, device=rows.device)
    if s["doc"] is not None:
        source = (T - (K - 1) + torch.arange(K - 1, device=rows.device)).clamp_min(0)
        keep = s["doc"][:, source] == s["doc"][:, T - 1:]
    return keep[..., None]


def _exact_conv_pass(s, back):
    x, w, rows, same = _exact_conv(s)
    T, K = x.shape[1], w.shape[1]
    pre = torch.zeros_like(x)
    for i in range(K):
        pre.addcmul_(rows[:, i:i + T] * same[:, :, i, None], w[:, i].expand_as(x))
    if s["b"] is not None:
        pre += s["b"].double()
    if not back:
        y = pre * torch.sigmoid(pre) if s["silu"] else pre
        return dict(y=y, state=rows[:, T:] * _exact_tail(s, rows, K))
    d = s["dy"].double()
    if s["silu"]:
        z = torch.sigmoid(pre)
        d = d * (z + pre * z * (1 - z))
    drows = torch.zeros_like(rows)
    dw = torch.zeros_like(w)
    for i in range(K):
        masked = d * same[:, :, i, None]
        dw[:, i] = torch.einsum("ntc,ntc->c", masked, rows[:, i:i + T])
        drows[:, i:i + T].addcmul_(masked, w[:, i].expand_as(x))
    if s["dstate"] is not None:
        drows[:, T:] += s["dstate"].double() * _exact_tail(s, rows, K)
    return dict(dx=drows[:, K - 1:], dw=dw, db=None if s["b"] is None else torch.einsum("ntc->c", d),
                dstate0=None if s["state"] is None else drows[:, :K - 1])


def _exact_ffn(s):
    x, W_in, W_out = s["x"].double(), s["W_in"].double(), s["W_out"].double()
    F = W_out.shape[0]
    gate = torch.nn.functional.silu if s["act"] == "silu" else torch.nn.functional.gelu
    if s["op"] == "ffn_fwd":
        gu = torch.matmul(x, W_in)
        y = torch.matmul(gate(gu[:, :F]).mul_(gu[:, F:]), W_out)
        return dict(y=y if s["residual"] is None else y + s["residual"].double(), gu=gu if s["save"] else None)
    dy = s["dy"].double()
    g = s["gu"][:, :F].double().requires_grad_()
    u = s["gu"][:, F:].double()
    with torch.enable_grad():
        a = gate(g)
    dh = torch.matmul(dy, W_out.transpose(0, 1))
    dg, = torch.autograd.grad(a, g, dh * u)
    a = a.detach()
    dgu = torch.cat((dg, dh * a), 1)
    return dict(dx=torch.matmul(dgu, W_in.transpose(0, 1)), dW_in=torch.matmul(x.transpose(0, 1), dgu),
                dW_out=torch.matmul((a * u).transpose(0, 1), dy))


def _exact_adamw(s):
    st, t = s["state"], int(s["state"]["step"][0]) + 1
    held = st["m"].numel()
    inside = torch.zeros(held, dtype=torch.bool, device="cuda")
    P, G = torch.zeros(held, dtype=torch.float64, device="cuda"), torch.zeros(held, dtype=torch.float64, device="cuda")
    for p, g, f in zip(s["params"], s["grads"], s["first"]):
        P[f:f + p.numel()], G[f:f + p.numel()] = p.double(), g.double()
        inside[f:f + p.numel()] = True
    if s["scale"] is not None:
        G *= s["scale"].double()
    eight = "m_scale" in st
    m, v = st["m"].double(), st["v"].double()
    if eight:
        m = (m.view(-1, BLOCK) * st["m_scale"].double()[:, None]).view(-1)
        v = (v.view(-1, BLOCK) * st["v_scale"].double()[:, None]).view(-1) ** 2
    m = torch.lerp(G, m, BETAS[0])
    v = torch.lerp(G * G, v, BETAS[1])
    hat = m / (1 - BETAS[0] ** t) / (torch.sqrt(v / (1 - BETAS[1] ** t)) + EPS)
    P = (P - LR * DECAY * P - LR * hat)[inside]
    # a moment in 8 bits goes up or down by the last bit of its 32-bit value: it has no value in 64 bits
    return dict(params=P, copies=None if s["copy"] is None else P, m=None if eight else m, v=None if eight else v,
                step=None)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("conv"):
        return _exact_conv_pass(s, s["op"] == "conv_bwd")
    if s["op"].startswith("ffn"):
        return _exact_ffn(s)
    return _exact_adamw(s)
