"""The operators around the memory scan: the gated linear recurrence with its gradient and
decode step, layer norm with its gradient, and the orthogonalised update.

    h, h_last = glr_fwd(x, g, h0=h0)
    d = glr_bwd(g, h, dh, h0=h0, dh_last=dh_last)        # d["dx"], d["dg"], d["dh0"]
    h = glr_step(x, g, state)                            # state updated in place
    y, mean, rstd = layer_norm_fwd(x, w, b)
    d = layer_norm_bwd(dy, x, mean, rstd, w)             # d["dx"], d["dw"], d["db"]
    O = orthogonalize(G)

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


def orthogonalize(G, *, coeffs=NS_COEFFS, eps=1e-7, out=None, workspace=None, stream=None):
    """Orthogonalised update of the matrices G ([..., m, n], fp32 or bf16, contiguous): one
    Newton-Schulz step X <- a X + (b A + c A^2) X, A = X X^T, per (a, b, c) of `coeffs`, from
    G / max(|G|_F, eps).  Returns bf16 [..., m, n]."""
    try:
        packed = b"".join(struct.pack("=3f", *step) for step in coeffs)
    except (TypeError, OverflowError, struct.error):
        raise TTMError(ERR_INVALID_ARG, "orthogonalize: coeffs is a sequence of (a, b, c) in fp32's range") from None
    return _call("orthogonalize", stream, G, packed, eps, out, workspace)


def _nothing(_key):
    return None
