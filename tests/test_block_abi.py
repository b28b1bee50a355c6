"""Host-side checks of the short convolution, the gated feed-forward block and AdamW, without a GPU: malformed
calls are rejected before anything is enqueued."""
import ctypes

import pytest

import test_neural_memory_gb300 as ttm
from tests.test_abi import P, host_only

INVALID, UNSUPPORTED = ttm.ERR_INVALID_ARG, ttm.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    ttm.build()
    return ttm.lib()


@host_only
def test_convolution_rejects_malformed(L):
    def fwd(N=2, T=4, C=16, K=4, dt=0, silu=1, x=P(0), xs=64, xt=16, w=P(1), b=P(2), s0=P(3), doc=P(4), ds=4, y=P(5), st=P(6)):
        return L.ttm_causal_conv_fwd(N, T, C, K, dt, silu, x, xs, xt, w, b, s0, doc, ds, y, st, None)
    assert fwd(N=0) == INVALID and fwd(T=-1) == INVALID and fwd(C=0) == INVALID and fwd(K=0) == INVALID
    assert fwd(dt=2) == INVALID and fwd(silu=2) == INVALID and fwd(x=None) == INVALID and fwd(w=None) == INVALID
    assert fwd(y=None) == INVALID and fwd(x=P(0, 2)) == INVALID and fwd(w=P(1, 2)) == INVALID
    assert fwd(s0=P(3, 8)) == INVALID and fwd(y=P(5, 4)) == INVALID and fwd(doc=P(4, 2)) == INVALID
    assert fwd(xt=15) == INVALID and fwd(xs=-64) == INVALID and fwd(xs=1 << 62) == INVALID and fwd(ds=-4) == INVALID
    assert fwd(y=P(0)) == INVALID and fwd(st=P(3)) == INVALID and fwd(st=P(5)) == INVALID and fwd(y=P(4)) == INVALID
    assert fwd(K=9) == UNSUPPORTED and fwd(N=1 << 20, C=1 << 12, T=0) == UNSUPPORTED
    assert fwd(N=1, T=2 ** 31 - 8192, C=1, xt=1, ds=2 ** 31) == UNSUPPORTED

    def bwd(dy=P(0), x=P(1), ds=P(5), dx=P(6), dw=P(7), db=P(8), d0=P(9), ws=P(10), wsb=1 << 20):
        return L.ttm_causal_conv_bwd(2, 4, 16, 4, 0, 1, dy, 64, 16, x, 64, 16, P(2), P(3), P(4), None, 0, ds, dx, dw, db, d0,
                                     ws, wsb, None)
    assert bwd(dy=None) == INVALID and bwd(dx=None) == INVALID and bwd(dx=P(1)) == INVALID and bwd(dw=P(8)) == INVALID
    assert bwd(d0=P(4)) == INVALID and bwd(ws=None) == INVALID and bwd(ws=P(6)) == INVALID and bwd(ds=P(5, 8)) == INVALID
    need = L.ttm_causal_conv_bwd_workspace_size(16, 4)
    assert need > 0 and bwd(wsb=need - 1) == INVALID
    assert L.ttm_causal_conv_bwd_workspace_size(0, 4) == 0 and L.ttm_causal_conv_bwd_workspace_size(16, 9) == 0

    def step(n=1, st=P(3), y=P(4)):
        return L.ttm_causal_conv_step(2, n, 16, 4, 0, 1, P(0), 64, 16, P(1), P(2), st, y, None)
    assert step(n=0) == INVALID and step(st=None) == INVALID and step(y=None) == INVALID and step(st=P(0)) == INVALID
    assert step(y=P(3)) == INVALID


@host_only
def test_feed_forward_rejects_malformed(L):
    need = L.ttm_gated_ffn_workspace_size(10, 64, 96, 0)
    back = L.ttm_gated_ffn_workspace_size(10, 64, 96, 1)
    assert need > 0 and back > 0

    def fwd(N=10, D=64, F=96, act=0, x=P(0), row=64, wi=P(1), wo=P(2), res=P(3), rr=64, y=P(4), gu=P(5), ws=P(6), wsb=1 << 20):
        return L.ttm_gated_ffn_fwd(N, D, F, act, x, row, wi, wo, res, rr, y, gu, ws, wsb, None)
    assert fwd(N=-1) == INVALID and fwd(D=0) == INVALID and fwd(D=60) == INVALID and fwd(F=4) == INVALID
    assert fwd(act=2) == INVALID and fwd(x=None) == INVALID and fwd(wi=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(row=63) == INVALID and fwd(row=68) == INVALID and fwd(rr=32) == INVALID and fwd(rr=76) == INVALID
    assert fwd(x=P(0, 8)) == INVALID and fwd(gu=P(5, 2)) == INVALID and fwd(y=P(3)) == INVALID and fwd(gu=P(1)) == INVALID
    assert fwd(ws=None) == INVALID and fwd(wsb=need - 1) == INVALID and fwd(ws=P(0)) == INVALID
    assert fwd(D=1 << 24, row=1 << 24) == UNSUPPORTED and fwd(N=2 ** 31 - 8000) == UNSUPPORTED

    def bwd(dy=P(0), dr=64, x=P(1), gu=P(2), dx=P(5), dwi=P(6), dwo=P(7), ws=P(8), wsb=1 << 20):
        return L.ttm_gated_ffn_bwd(10, 64, 96, 0, dy, dr, x, 64, gu, P(3), P(4), dx, dwi, dwo, ws, wsb, None)
    assert bwd(dy=None) == INVALID and bwd(dr=60) == INVALID and bwd(gu=None) == INVALID and bwd(dx=P(1)) == INVALID
    assert bwd(dwi=P(7)) == INVALID and bwd(wsb=back - 1) == INVALID and bwd(ws=P(2)) == INVALID
    assert L.ttm_gated_ffn_workspace_size(10, 60, 96, 0) == 0 and L.ttm_gated_ffn_workspace_size(0, 64, 96, 0) == 0


class Entry(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("n", ctypes.c_longlong),
                ("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int)]


@host_only
def test_adamw_rejects_malformed(L):
    def call(entries=((P(0), P(1), P(2), 300, 0, 0),), bits=32, m=P(10), v=P(11), ms=None, vs=None, step=P(12), lr=0.1, lr_at=None,
             b1=0.9, b2=0.9, eps=1e-8, wd=0.0, gs=None, count=None):
        arr = (Entry * max(1, len(entries)))(*[Entry(*e) for e in entries])
        return L.ttm_adamw_step(len(entries) if count is None else count, arr, bits, m, v, ms, vs, step, lr, lr_at, b1, b2, eps,
                                wd, gs, None)
    one = lambda **k: call(entries=(tuple({**dict(p=P(0), g=P(1), c=P(2), n=300, pd=0, gd=0), **k}.values()),))  # noqa: E731
    assert call(count=-1) == INVALID and call(bits=16) == INVALID and call(step=None) == INVALID and call(m=None) == INVALID
    assert call(b1=1.0) == INVALID and call(b2=-0.5) == INVALID and call(eps=0.0) == INVALID and call(eps=1e-60) == INVALID
    assert call(lr=float("inf")) == INVALID and call(wd=float("nan")) == INVALID
    assert call(bits=8) == INVALID and call(ms=P(20), vs=P(21)) == INVALID and call(bits=8, ms=P(20)) == INVALID
    assert call(m=P(10, 8)) == INVALID and call(step=P(12, 2)) == INVALID and call(gs=P(13, 1)) == INVALID
    assert one(n=1 << 41) == UNSUPPORTED and one(n=1 << 62) == UNSUPPORTED
    assert one(p=None) == INVALID and one(n=-1) == INVALID and one(pd=3) == INVALID and one(gd=2) == INVALID
    assert one(p=P(0, 2)) == INVALID and one(g=P(1, 1)) == INVALID and one(c=P(2, 1)) == INVALID
    assert one(g=P(0)) == INVALID and one(c=P(0)) == INVALID and one(p=P(10)) == INVALID and one(g=P(11, 64)) == INVALID
    assert call(v=P(10)) == INVALID and call(step=P(10)) == INVALID and call(gs=P(0)) == INVALID and call(lr_at=P(12)) == INVALID
    twice = ((P(0), P(1), None, 300, 0, 0), (P(0, 1196), P(1), None, 300, 0, 0))
    assert call(entries=twice) == INVALID
    assert L.ttm_adamw_moments(-1, P(0), P(1), P(2), P(3), P(4), P(5), None) == INVALID
    assert L.ttm_adamw_moments(4, P(0), P(1), P(2), P(3), P(4), P(4), None) == INVALID
    assert L.ttm_adamw_moments(4, P(0), None, P(2), P(3), P(4), P(5), None) == INVALID
