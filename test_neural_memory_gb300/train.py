"""The operators around the memory scan: the gated linear recurrence with its gradient and
decode step, layer norm with its gradient, the short causal convolution with its gradient and
decode step, the gated feed-forward block with its gradient, the orthogonalised update and AdamW.

    h, h_last = glr_fwd(x, g, h0=h0)
    d = glr_bwd(g, h, dh, h0=h0, dh_last=dh_last)        # d["dx"], d["dg"], d["dh0"]
    h = glr_step(x, g, state)                            # state updated in place
    y, mean, rstd = layer_norm_fwd(x, w, b)
    d = layer_norm_bwd(dy, x, mean, rstd, w)             # d["dx"], d["dw"], d["db"]
    y, state = causal_conv_fwd(x, w, b)                  # state: the last inputs
    d = causal_conv_bwd(dy, x, w, b)                     # d["dx"], d["dw"], d["db"], d["dstate0"]
    y = causal_conv_step(x, w, state, b)                 # state updated in place
    y, gu = gated_ffn_fwd(x, W_in, W_out, residual=r)
    d = gated_ffn_bwd(dy, x, gu, W_in, W_out)            # d["dx"], d["dW_in"], d["dW_out"]
    O = orthogonalize(G)
    state = adamw_state(params, bits=8)
    adamw_step(params, grads, state, lr=1e-3)            # params and state updated in place

As elsewhere in the package the arguments are only checked and marshalled on the way to the
library (csrc/bind_train.cpp, compiled because these calls are short); outputs and workspaces
are allocated with torch when not given.  A call runs on the current stream of its tensors'
device, or on `stream`, which then also owns what the call allocates.  Malformed arguments
raise TTMError (ERR_INVALID_ARG, or ERR_UNSUPPORTED for sizes beyond the library's), other
dtypes than float32 and bfloat16 TypeError.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
import struct

import torch

from . import ERR_INVALID_ARG, TTMError, lib
from ._build import BIND

# (a, b, c) of the five default steps of orthogonalize: the quintic of the Muon optimiser, which
# takes singular values to about 0.7 .. 1.2, small ones by a factor of 3.4 a step.
NS_COEFFS = ((3.4445, -4.7750, 2.0315),) * 5

ACTS = {"silu": 0, "gelu": 1}

_bind = None


def _load():
    global _bind
    lib()                                    # raises if the library has not been built
    if not os.path.exists(BIND):
        raise RuntimeError(f"{BIND} is missing; build it with "
                           "`python -m test_neural_memory_gb300._build`")
    loader = importlib.machinery.ExtensionFileLoader("ttm_torch", BIND)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("ttm_torch", loader))
    loader.exec_module(module)
    module.set_error(TTMError)
    _bind = module
    return module


def _call(name, stream, *args):
    f = getattr(_bind or _load(), name)
    if stream is None:
        return f(*args)
    with torch.cuda.stream(stream):
        return f(*args)


def glr_fwd(x, g, *, h0=None, h=None, h_last=None, workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over the tokens of x
    ([..., T, D], fp32 or bf16; may be a column slice).  g: the log of the retention, one
    value per channel (shape and dtype of x) or per token ([..., T] fp32).  h0: [..., D]
    fp32 or None.  Returns (h like x, h_last [..., D] fp32)."""
    return _call("glr_fwd", stream, x, g, h0, h, h_last, workspace)


def glr_bwd(g, h, dh, *, h0=None, dh_last=None, want_dh0=True, workspace=None, out=None,
            stream=None):
    """Gradient of glr_fwd: h is what the forward call returned, dh ([..., T, D]) and dh_last
    ([..., D] fp32 or None) the adjoints of its outputs.  Returns a dict with dx, dg (shaped
    as x and g) and dh0 ([..., D] fp32, None when want_dh0 is False).  `out` may hold
    preallocated tensors for these keys."""
    o = out.get if out else _nothing
    dx, dg, dh0 = _call("glr_bwd", stream, g, h, dh, h0, dh_last, bool(want_dh0), o("dx"), o("dg"),
                        o("dh0"), workspace)
    return dict(dx=dx, dg=dg, dh0=dh0)


def glr_step(x, g, state, *, h=None, stream=None):
    """Decode step of the recurrence: continues every sequence by the n tokens of x
    ([..., n, D]) from `state` ([..., D] fp32, updated in place).  g as in glr_fwd.
    Returns h like x."""
    return _call("glr_step", stream, x, g, state, h)


def layer_norm_fwd(x, w=None, b=None, *, eps=1e-5, y=None, mean=None, rstd=None, want_stats=True,
                   stream=None):
    """Layer norm over the last axis of x ([..., D], fp32 or bf16; rows may be slices of wider
    ones); w, b: [D] fp32 or None.  Returns (y, mean, rstd), the statistics [...] fp32 for
    layer_norm_bwd (None when want_stats is False)."""
    return _call("layer_norm_fwd", stream, x, w, b, eps, y, mean, rstd, bool(want_stats))


def layer_norm_bwd(dy, x, mean, rstd, w=None, *, want_dw=True, want_db=True, workspace=None,
                   out=None, stream=None):
    """Gradient of layer_norm_fwd for the adjoint dy of y; x, w: its inputs, mean, rstd: the
    statistics it returned.  Returns a dict with dx (like x) and dw, db ([D] fp32, summed over
    the rows; None when not wanted).  `out` may hold preallocated tensors for these keys."""
    o = out.get if out else _nothing
    dx, dw, db = _call("layer_norm_bwd", stream, dy, x, mean, rstd, w, bool(want_dw), bool(want_db),
                       o("dx"), o("dw"), o("db"), workspace)
    return dict(dx=dx, dw=dw, db=db)


def causal_conv_fwd(x, w, b=None, *, state0=None, doc=None, silu=True, want_state=True, y=None, state=None,
                    stream=None):
    """Depthwise causal convolution over the tokens of x ([..., T, C], fp32 or bf16; may be a column
    slice) with the K <= 8 taps of w ([C, K] fp32, the last one the token's own) and b ([C] fp32 or
    None), then SiLU unless silu is False.  state0: the K - 1 inputs before the first token ([..., K-1, C]
    in the dtype of x) or None (zero).  doc ([..., T] int32): taps of another document's rows are left
    out.  Returns (y like x, state [..., K-1, C]): state continues the sequences (None when
    want_state is False)."""
    return _call("causal_conv_fwd", stream, x, w, b, state0, doc, bool(silu), bool(want_state), y, state)


def causal_conv_bwd(dy, x, w, b=None, *, state0=None, doc=None, silu=True, dstate=None, want_dw=True,
                    workspace=None, out=None, stream=None):
    """Gradient of causal_conv_fwd for the adjoints dy of y and dstate of state (or None); the rest as in the
    forward call.  Returns a dict with dx (like x), dw ([C, K] fp32), db ([C] fp32, None without b;
    both None when want_dw is False) and dstate0 (like state0, None without it).  `out` may hold
    preallocated tensors for these keys."""
    o = out.get if out else _nothing
    dx, dw, db, ds = _call("causal_conv_bwd", stream, dy, x, w, b, state0, doc, bool(silu), dstate, bool(want_dw),
                           o("dx"), o("dw"), o("db"), o("dstate0"), workspace)
    return dict(dx=dx, dw=dw, db=db, dstate0=ds)


def causal_conv_step(x, w, state, b=None, *, silu=True, y=None, stream=None):
    """Decode step of the convolution: continues every sequence by the n tokens of x ([..., n, C]) from
    `state` ([..., K-1, C] in the dtype of x, updated in place).  For few tokens (they are walked one after the
    other): a long continuation is causal_conv_fwd's with state0.  Returns y like x."""
    return _call("causal_conv_step", stream, x, w, state, b, bool(silu), y)


def gated_ffn_fwd(x, W_in, W_out, *, act="silu", residual=None, want_gu=True, y=None, gu=None, workspace=None,
                  stream=None):
    """Gated feed-forward block y = (act(x W_g) * (x W_u)) W_out (+ residual), all bf16, widths multiples
    of 8.  x: [..., D] (rows may be slices of wider ones); W_in: [D, 2F], W_g then W_u; W_out: [F, D];
    act: "silu" or "gelu" (erf).  Returns (y like x, gu [..., 2F]): what gated_ffn_bwd takes (None
    when want_gu is False)."""
    return _call("gated_ffn_fwd", stream, x, W_in, W_out, _act(act), residual, bool(want_gu), y, gu, workspace)


def gated_ffn_bwd(dy, x, gu, W_in, W_out, *, act="silu", want_dx=True, want_dw=True, workspace=None, out=None,
                  stream=None):
    """Gradient of gated_ffn_fwd for the adjoint dy of y; gu: what the forward call returned (the
    residual's adjoint is dy).  Returns a dict with dx, dW_in, dW_out (bf16, like x and the weights; None
    when not wanted).  `out` may hold preallocated tensors for these keys."""
    o = out.get if out else _nothing
    dx, dW_in, dW_out = _call("gated_ffn_bwd", stream, dy, x, gu, W_in, W_out, _act(act), bool(want_dx),
                              bool(want_dw), o("dx"), o("dW_in"), o("dW_out"), workspace)
    return dict(dx=dx, dW_in=dW_in, dW_out=dW_out)


def adamw_state(params, *, bits=32):
    """Fresh moments for adamw_step: a dict of tensors on the device of `params` (which may be saved and
    loaded as they are).  m, v: flat, the moments of params[i] from value 256 * (256-value blocks of the
    tensors before it) on; fp32, or for bits=8 float8_e4m3fn (v then holds the square root) with m_scale,
    v_scale, a power of two per 256 values.  step: int32 [2], the steps done and an internal zero."""
    params = list(params)
    if bits not in (8, 32):
        raise TTMError(ERR_INVALID_ARG, "adamw_state: bits is 8 or 32")
    if not params:
        raise TTMError(ERR_INVALID_ARG, "adamw_state: no parameters")
    dev, blocks = params[0].device, sum((p.numel() + 255) // 256 for p in params)
    zeros = lambda n, t: torch.zeros(n, dtype=t, device=dev)  # noqa: E731
    state = {k: zeros(blocks * 256, torch.float32 if bits == 32 else torch.float8_e4m3fn) for k in ("m", "v")}
    if bits == 8:
        state.update({k: zeros(blocks, torch.float32) for k in ("m_scale", "v_scale")})
    state["step"] = zeros(2, torch.int32)
    return state


def adamw_step(params, grads, state, *, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, grad_scale=None,
               copies=None, stream=None):
    """AdamW step over many tensors in one pass, params (fp32 or bf16, contiguous) and `state` (from
    adamw_state for the same tensors in the same order) updated in place.  bf16 params are rounded to nearest and stand still
    under steps below 2^-9 of them; fp32 params with copies do not.  grads: fp32 or bf16, None leaves its
    parameter and moments as they are.  copies: None, or bf16 tensors (or None) written with the new
    values.  lr: a number, or a 0-dim fp32 tensor on the device; grad_scale: a 0-dim fp32 tensor that
    multiplies the gradients, or None.  The steps are counted on the device, so that a captured
    call counts its replays."""
    try:
        m, v, step = state["m"], state["v"], state["step"]
        b1, b2 = betas
    except (TypeError, ValueError, KeyError):
        raise TTMError(ERR_INVALID_ARG, "adamw_step: state comes from adamw_state, betas are two numbers") from None
    _call("adamw_step", stream, params, grads, copies, m, v, state.get("m_scale"), state.get("v_scale"), step, lr, b1, b2,
          eps, weight_decay, grad_scale)


def adamw_moments(state, *, stream=None):
    """(m, v) of adamw_state's dict in fp32, laid out as there: its own tensors for 32 bits, new ones for 8."""
    if "m_scale" not in state:
        return state["m"], state["v"]
    return _call("adamw_moments", stream, state["m"], state["v"], state["m_scale"], state["v_scale"])


def orthogonalize(G, *, coeffs=NS_COEFFS, eps=1e-7, out=None, workspace=None, stream=None):
    """Orthogonalised update of the matrices G ([..., m, n], fp32 or bf16, contiguous): one
    Newton-Schulz step X <- a X + (b A + c A^2) X, A = X X^T, per (a, b, c) of `coeffs`, from
    G / max(|G|_F, eps).  Returns bf16 [..., m, n]."""
    try:
        packed = b"".join(struct.pack("=3f", *step) for step in coeffs)
    except (TypeError, OverflowError, struct.error):
        raise TTMError(ERR_INVALID_ARG, "orthogonalize: coeffs is a sequence of (a, b, c) in fp32's range") from None
    return _call("orthogonalize", stream, G, packed, eps, out, workspace)


def _act(name):
    if name not in ACTS:
        raise TTMError(ERR_INVALID_ARG, 'act is "silu" or "gelu"')
    return ACTS[name]


def _nothing(_key):
    return None
