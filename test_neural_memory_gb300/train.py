"""Binding of the operators around the memory scan: the gated linear recurrence with its
gradient and decode step, layer norm with its gradient, and the orthogonalised update.

    h, h_last = glr_fwd(x, g, h0=h0)
    d = glr_bwd(g, h, dh, h0=h0, dh_last=dh_last)        # d["dx"], d["dg"], d["dh0"]
    h = glr_step(x, g, state)                            # state updated in place
    y, mean, rstd = layer_norm_fwd(x, w, b)
    d = layer_norm_bwd(dy, x, mean, rstd, w)             # d["dx"], d["dw"], d["db"]
    O = orthogonalize(G)

As elsewhere in the package only arguments are marshalled here; outputs and workspaces
are allocated with torch (on the call's stream) when not given.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import BF16, ERR_INVALID_ARG, F32, OK, TTMError, lib

GATE_CHANNEL, GATE_TOKEN = 0, 1
_CODES = {torch.float32: F32, torch.bfloat16: BF16}

# (a, b, c) of the five default steps of orthogonalize: the quintic of the Muon optimiser,
# which takes singular values between about 1e-3 and 1 to the range 0.7 .. 1.2.
NS_COEFFS = ((3.4445, -4.7750, 2.0315),) * 5


def _bad(what):
    raise TTMError(ERR_INVALID_ARG, what)


def _code(t, what):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return code


def _done(code, what):
    if code != OK:
        raise TTMError(code, what)


def _raw(t, stream):
    """The call's stream as CUDA sees it: `stream`, or the current one of t's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream


def _on(stream):
    """Allocations inside belong to the stream the call runs on."""
    return _HERE if stream is None else torch.cuda.stream(stream)


_HERE = contextlib.nullcontext()
_F32, _BF16 = torch.float32, torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


def _f32(t, shape, device, what):
    """Checks a contiguous fp32 tensor (or None) of the given shape on the call's device."""
    if t is not None and (t.dtype is not _F32 or t.shape != shape or not t.is_contiguous() or
                          t.device != device):
        _bad(f"{what} must be a contiguous float32 tensor of shape {tuple(shape)}")


def _out(t, shape, dtype, device, what):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        _bad(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


def _out_like(t, x, what):
    """An output of the shape and dtype of x, contiguous."""
    if t is None and x.is_contiguous():
        return torch.empty_like(x)
    return _out(t, x.shape, x.dtype, x.device, what)


def _scratch(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if workspace.device != device or not workspace.is_contiguous():
        _bad("workspace must be a contiguous tensor on the device of the call")
    return workspace


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _one_stride(shape, st, lead, what):
    """Elements between consecutive entries of the first `lead` dimensions taken as one;
    None when there is at most one entry."""
    step, size = None, 1
    for k in range(lead - 1, -1, -1):
        if shape[k] == 1:
            continue
        if step is None:
            step = st[k]
        elif st[k] != step * size:
            _bad(f"{what}: the leading dimensions {tuple(shape[:lead])} have no single stride")
        size *= shape[k]
    return step


def _strides(t, lead, inner, what):
    """(sequence stride, token stride) in elements of a view whose first `lead` dimensions
    number the sequences and whose next one the tokens of `inner` values."""
    shape, st = t.shape, t.stride()
    if lead == 1 and shape[0] > 1 and shape[1] > 1:
        return st[0], st[1]
    tok = st[lead] if shape[lead] > 1 else inner
    seq = _one_stride(shape, st, lead, what)
    return shape[lead] * tok if seq is None else seq, tok


def _glr_shapes(x, g, what):
    """Common checks: x [..., T, D], g of the same shape (a gate per channel, x's dtype) or
    [..., T] (a gate per token, fp32).  Returns (shape of the state, N, T, D, dtype code, gate
    code, x's sequence and token stride, g's sequence and token stride)."""
    shape = x.shape
    lead = len(shape) - 2
    if lead < 0:
        _bad(f"{what}: expected [..., T, D]")
    if lead == 1:
        N, T, D = shape
        state = (N, D)
    else:
        T, D = shape[-2:]
        state, N = (*shape[:-2], D), 1
        for s in shape[:-2]:
            N *= s
    dt = _code(x, what)
    if (D > 1 and x.stride(-1) != 1) or not x.is_cuda or x.device != g.device:
        _bad(f"{what}: channels must be contiguous, all tensors on one CUDA device")
    gshape = g.shape
    if len(gshape) == lead + 2:
        if gshape != shape or g.dtype is not x.dtype or (D > 1 and g.stride(-1) != 1):
            _bad(f"{what}: a gate per channel has the shape, dtype and channel order of x")
        gate, inner = GATE_CHANNEL, D
    else:
        if gshape != shape[:-1] or g.dtype is not _F32:
            _bad(f"{what}: a gate per token is float32 of shape {tuple(shape[:-1])}")
        gate, inner = GATE_TOKEN, 1
    return (state, N, T, D, dt, gate, *_strides(x, lead, D, what), *_strides(g, lead, inner, what))


def glr_fwd(x, g, *, h0=None, h=None, h_last=None, workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over the tokens of x
    ([..., T, D], fp32 or bf16; may be a column slice).  g: the log of the retention, one
    value per channel (shape and dtype of x) or per token ([..., T] fp32).  h0: [..., D]
    fp32 or None.  Returns (h like x, h_last [..., D] fp32)."""
    state, N, T, D, dt, gate, xs, xt, gs, gt = _glr_shapes(x, g, "glr_fwd")
    dev, L = x.device, lib()
    _f32(h0, state, dev, "h0")
    with _on(stream):
        h = _out_like(h, x, "h")
        h_last = _out(h_last, state, _F32, dev, "h_last")
        workspace = _scratch(workspace, L.ttm_glr_workspace_size(N, T, D, dt, gate, 0), dev)
    _done(L.ttm_glr_fwd(N, T, D, dt, gate, x.data_ptr(), xs, xt, g.data_ptr(), gs, gt, _p(h0),
                        h.data_ptr(), h_last.data_ptr(), _p(workspace), _nbytes(workspace),
                        _raw(x, stream)), "ttm_glr_fwd")
    return h, h_last


def glr_bwd(g, h, dh, *, h0=None, dh_last=None, want_dh0=True, workspace=None, out=None,
            stream=None):
    """Gradient of glr_fwd: h is what the forward call returned, dh ([..., T, D]) and dh_last
    ([..., D] fp32 or None) the adjoints of its outputs.  Returns a dict with dx, dg (shaped
    as x and g) and dh0 ([..., D] fp32, None when want_dh0 is False).  `out` may hold
    preallocated tensors for these keys."""
    state, N, T, D, dt, gate, ds, dtok, gs, gt = _glr_shapes(dh, g, "glr_bwd")
    dev, L = dh.device, lib()
    if h.shape != dh.shape or h.dtype is not dh.dtype or not h.is_contiguous() or h.device != dev:
        _bad("glr_bwd: h must be contiguous, of the shape and dtype of dh")
    _f32(h0, state, dev, "h0")
    _f32(dh_last, state, dev, "dh_last")
    out = out or {}
    with _on(stream):
        dx = _out_like(out.get("dx"), dh, "dx")
        dg = _out_like(out.get("dg"), g, "dg")
        dh0 = _out(out.get("dh0"), state, _F32, dev, "dh0") if want_dh0 else None
        workspace = _scratch(workspace, L.ttm_glr_workspace_size(N, T, D, dt, gate, 1), dev)
    _done(L.ttm_glr_bwd(N, T, D, dt, gate, g.data_ptr(), gs, gt, h.data_ptr(), _p(h0),
                        dh.data_ptr(), ds, dtok, _p(dh_last), dx.data_ptr(), dg.data_ptr(),
                        _p(dh0), _p(workspace), _nbytes(workspace), _raw(dh, stream)),
          "ttm_glr_bwd")
    return dict(dx=dx, dg=dg, dh0=dh0)


def glr_step(x, g, state, *, h=None, stream=None):
    """Decode step of the recurrence: continues every sequence by the n tokens of x
    ([..., n, D]) from `state` ([..., D] fp32, updated in place).  g as in glr_fwd.
    Returns h like x."""
    shape, N, n, D, dt, gate, xs, xt, gs, gt = _glr_shapes(x, g, "glr_step")
    if state is None:
        _bad("glr_step: state is required")
    _f32(state, shape, x.device, "state")
    with _on(stream):
        h = _out_like(h, x, "h")
    _done(lib().ttm_glr_step(N, n, D, dt, gate, x.data_ptr(), xs, xt, g.data_ptr(), gs, gt,
                             state.data_ptr(), h.data_ptr(), _raw(x, stream)), "ttm_glr_step")
    return h


def _ln_rows(x, what):
    """Number of rows and elements between them of x [..., D] with contiguous last axis."""
    if x.dim() < 1 or (x.shape[-1] > 1 and x.stride(-1) != 1) or not x.is_cuda:
        _bad(f"{what}: expected a CUDA tensor [..., D] with a contiguous last axis")
    D, N = x.shape[-1], 1
    for s in x.shape[:-1]:
        N *= s
    if x.is_contiguous():
        return N, D
    row = _one_stride(x.shape, x.stride(), x.dim() - 1, what)
    return N, D if row is None else row


def layer_norm_fwd(x, w=None, b=None, *, eps=1e-5, y=None, mean=None, rstd=None, want_stats=True,
                   stream=None):
    """Layer norm over the last axis of x ([..., D], fp32 or bf16; rows may be slices of wider
    ones); w, b: [D] fp32 or None.  Returns (y, mean, rstd), the statistics [...] fp32 for
    layer_norm_bwd (None when want_stats is False)."""
    N, row = _ln_rows(x, "layer_norm_fwd")
    D, dev, dt = x.shape[-1], x.device, _code(x, "x")
    _f32(w, (D,), dev, "w")
    _f32(b, (D,), dev, "b")
    with _on(stream):
        y = _out_like(y, x, "y")
        if want_stats:
            mean = _out(mean, x.shape[:-1], _F32, dev, "mean")
            rstd = _out(rstd, x.shape[:-1], _F32, dev, "rstd")
        else:
            mean = rstd = None
    _done(lib().ttm_layer_norm_fwd(N, D, dt, x.data_ptr(), row, _p(w), _p(b), eps, y.data_ptr(),
                                   _p(mean), _p(rstd), _raw(x, stream)), "ttm_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, w=None, *, want_dw=True, want_db=True, workspace=None,
                   out=None, stream=None):
    """Gradient of layer_norm_fwd for the adjoint dy of y; x, w: its inputs, mean, rstd: the
    statistics it returned.  Returns a dict with dx (like x) and dw, db ([D] fp32, summed over
    the rows; None when not wanted).  `out` may hold preallocated tensors for these keys."""
    N, row = _ln_rows(x, "layer_norm_bwd")
    D, dev, dt = x.shape[-1], x.device, _code(x, "x")
    if dy.shape != x.shape or dy.dtype is not x.dtype or dy.device != dev:
        _bad("layer_norm_bwd: dy must have the shape and dtype of x")
    _, dy_row = _ln_rows(dy, "layer_norm_bwd")
    if mean is None or rstd is None:
        _bad("layer_norm_bwd: mean and rstd are required")
    _f32(mean, x.shape[:-1], dev, "mean")
    _f32(rstd, x.shape[:-1], dev, "rstd")
    _f32(w, (D,), dev, "w")
    out, L = out or {}, lib()
    with _on(stream):
        dx = _out_like(out.get("dx"), x, "dx")
        dw = _out(out.get("dw"), (D,), _F32, dev, "dw") if want_dw else None
        db = _out(out.get("db"), (D,), _F32, dev, "db") if want_db else None
        need = L.ttm_layer_norm_bwd_workspace_size(N, D) if want_dw or want_db else 0
        workspace = _scratch(workspace, need, dev)
    _done(L.ttm_layer_norm_bwd(N, D, dt, dy.data_ptr(), dy_row, x.data_ptr(), row, _p(w),
                               mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _p(dw), _p(db),
                               _p(workspace), _nbytes(workspace), _raw(x, stream)),
          "ttm_layer_norm_bwd")
    return dict(dx=dx, dw=dw, db=db)


def orthogonalize(G, *, coeffs=NS_COEFFS, eps=1e-7, out=None, workspace=None, stream=None):
    """Orthogonalised update of the matrices G ([..., m, n], fp32 or bf16, contiguous): one
    Newton-Schulz step X <- a X + (b A + c A^2) X, A = X X^T, per (a, b, c) of `coeffs`, from
    G / max(|G|_F, eps).  Returns bf16 [..., m, n]."""
    dt, dev, L = _code(G, "G"), G.device, lib()
    if G.dim() < 2 or not G.is_contiguous() or not G.is_cuda:
        _bad("orthogonalize: expected a contiguous CUDA tensor [..., m, n]")
    m, n = G.shape[-2:]
    batch = 1
    for s in G.shape[:-2]:
        batch *= s
    flat = [float(v) for step in coeffs for v in step]
    if len(flat) != 3 * len(coeffs):
        _bad("orthogonalize: coeffs is a sequence of (a, b, c)")
    with _on(stream):
        out = _out(out, G.shape, torch.bfloat16, dev, "out")
        workspace = _scratch(workspace, L.ttm_orthogonalize_workspace_size(batch, m, n), dev)
    _done(L.ttm_orthogonalize(batch, m, n, dt, G.data_ptr(), (ctypes.c_float * len(flat))(*flat),
                              len(coeffs), eps, out.data_ptr(), _p(workspace), _nbytes(workspace),
                              _raw(G, stream)), "ttm_orthogonalize")
    return out
