"""Host-side checks of the operators around the scan, without a GPU: malformed calls are
rejected before anything is enqueued, and the workspace sizes."""
import ctypes

import pytest

import test_neural_memory_gb300 as ttm
from tests.test_abi import P, host_only

INVALID, UNSUPPORTED = ttm.ERR_INVALID_ARG, ttm.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    ttm.build()
    return ttm.lib()


def glr(L, N=2, T=4, D=16, dt=0, gate=0, x=P(0), xs=64, xt=16, g=P(1), gs=64, gt=16, h0=None,
        h=P(2), last=P(3), ws=P(4), wsb=1 << 18):
    return L.ttm_glr_fwd(N, T, D, dt, gate, x, xs, xt, g, gs, gt, h0, h, last, ws, wsb, None)


@host_only
def test_recurrence_rejects_malformed(L):
    assert glr(L, N=0) == INVALID and glr(L, T=-1) == INVALID and glr(L, D=0) == INVALID
    assert glr(L, dt=2) == INVALID and glr(L, gate=2) == INVALID
    assert glr(L, x=None) == INVALID and glr(L, g=None) == INVALID
    assert glr(L, h=None) == INVALID and glr(L, last=None) == INVALID
    assert glr(L, x=P(0, 2)) == INVALID              # fp32 values at half a word
    assert glr(L, h=P(2, 8)) == INVALID and glr(L, last=P(3, 4)) == INVALID
    assert glr(L, xt=15) == INVALID                  # tokens overlap
    assert glr(L, xs=15) == INVALID and glr(L, gs=-64) == INVALID
    assert glr(L, xs=1 << 62) == INVALID             # offsets beyond 64 bits
    assert glr(L, h=P(0)) == INVALID and glr(L, last=P(1)) == INVALID
    assert glr(L, h0=P(3)) == INVALID                # h_last over h0
    assert glr(L, ws=P(2)) == INVALID                # workspace over an output
    assert glr(L, N=1 << 20, D=1 << 12, T=0) == UNSUPPORTED
    r = L.ttm_glr_bwd(2, 4, 16, 0, 0, P(0), 64, 16, P(1), None, P(2), 64, 16, None, P(3), P(3), None,
                      P(5), 1 << 18, None)
    assert r == INVALID                              # dg over dx
    r = L.ttm_glr_bwd(2, 4, 16, 0, 0, P(0), 64, 16, None, None, P(2), 64, 16, None, P(3), P(4), None,
                      P(5), 1 << 18, None)
    assert r == INVALID                              # the forward's h is missing
    r = L.ttm_glr_step(2, 0, 16, 0, 0, P(0), 64, 16, P(1), 64, 16, P(2), P(3), None)
    assert r == INVALID                              # a step of no tokens
    r = L.ttm_glr_step(2, 1, 16, 0, 0, P(0), 64, 16, P(1), 64, 16, P(0), P(3), None)
    assert r == INVALID                              # state over x


@host_only
def test_recurrence_needs_its_workspace(L):
    need = L.ttm_glr_workspace_size(2, 100000, 64, 1, 0, 0)
    if need:
        assert glr(L, T=100000, D=64, dt=1, xs=6400000, xt=64, gs=6400000, gt=64, g=P(100),
                   h=P(200), last=P(300), ws=P(400), wsb=need - 1) == INVALID
    assert L.ttm_glr_workspace_size(0, 1, 1, 0, 0, 0) == 0
    assert L.ttm_glr_workspace_size(1, 1, 1, 7, 0, 0) == 0


@host_only
def test_layer_norm_rejects_malformed(L):
    def fwd(N=4, D=16, dt=0, x=P(0), row=16, w=P(1), b=P(2), eps=1e-5, y=P(3), mean=P(4), rstd=P(5)):
        return L.ttm_layer_norm_fwd(N, D, dt, x, row, w, b, eps, y, mean, rstd, None)
    assert fwd(N=-1) == INVALID and fwd(D=0) == INVALID and fwd(dt=3) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(row=15) == INVALID
    assert fwd(w=P(1, 4)) == INVALID and fwd(y=P(0)) == INVALID and fwd(mean=P(3)) == INVALID

    def bwd(N=4, D=16, dy=P(0), x=P(1), w=P(2), mean=P(3), rstd=P(4), dx=P(5), dw=P(6), db=P(7),
            ws=P(8), wsb=1 << 20):
        return L.ttm_layer_norm_bwd(N, D, 0, dy, 16, x, 16, w, mean, rstd, dx, dw, db, ws, wsb, None)
    assert bwd(mean=None) == INVALID and bwd(dx=None) == INVALID and bwd(dx=P(1)) == INVALID
    assert bwd(dw=P(7)) == INVALID and bwd(ws=None) == INVALID and bwd(ws=P(5)) == INVALID
    assert bwd(wsb=L.ttm_layer_norm_bwd_workspace_size(4, 16) - 1) == INVALID
    assert L.ttm_layer_norm_bwd_workspace_size(4, 0) == 0


@host_only
def test_orthogonalize_rejects_malformed(L):
    def call(batch=1, m=20, n=30, dt=0, G=P(0), c=(3.0, -4.0, 2.0), steps=None, eps=1e-7, out=P(1),
             ws=P(2), wsb=1 << 20):
        arr = (ctypes.c_float * max(1, len(c)))(*c)
        return L.ttm_orthogonalize(batch, m, n, dt, G, arr, len(c) // 3 if steps is None else steps,
                                   eps, out, ws, wsb, None)
    assert call(batch=0) == INVALID and call(m=0) == INVALID and call(n=0) == INVALID
    assert call(dt=9) == INVALID and call(G=None) == INVALID and call(out=None) == INVALID
    assert call(steps=-1) == INVALID and call(eps=0.0) == INVALID
    assert call(c=(1.0, float("nan"), 1.0)) == INVALID and call(c=(1.0, 1.0, 1.0) * 33) == UNSUPPORTED
    assert call(m=1 << 17) == UNSUPPORTED and call(batch=1 << 17) == UNSUPPORTED
    assert call(G=P(0, 8)) == INVALID and call(out=P(0)) == INVALID and call(ws=P(1)) == INVALID
    need = L.ttm_orthogonalize_workspace_size(1, 300, 400)
    assert need > 0 and call(m=300, n=400, wsb=need - 1) == INVALID
    assert L.ttm_orthogonalize_workspace_size(1, 0, 4) == 0


@host_only
def test_recurrence_refuses_lengths_its_tiles_cannot_count(L):
    for T in (2 ** 31 - 1, 2 ** 31 - 8192):
        assert glr(L, N=1, T=T, D=1, xt=1, gt=1) == UNSUPPORTED
        assert L.ttm_glr_workspace_size(1, T, 1, 0, 0, 0) == 0
        assert L.ttm_glr_step(1, T, 1, 0, 0, P(0), 0, 1, P(1), 0, 1, P(2), P(3), None) == UNSUPPORTED
        assert L.ttm_glr_bwd(1, T, 1, 0, 0, P(0), 0, 1, P(1), None, P(2), 0, 1, None, P(3), P(4), None,
                             P(5), 1 << 18, None) == UNSUPPORTED
    assert L.ttm_glr_workspace_size(1, 2 ** 31 - 8193, 1, 0, 0, 0) > 0


@pytest.mark.parametrize("coeffs", [[(1.0, 2.0), (3.0, 4.0, 5.0, 6.0)], [1.0, 2.0, 3.0], [(1.0, 2.0, "3")], 7.0,
                                    [(1.0, 2.0, 1e300)]])
def test_coefficients_come_in_threes(coeffs):
    with pytest.raises(ttm.TTMError, match="coeffs") as e:
        ttm.orthogonalize(None, coeffs=coeffs)
    assert e.value.code == INVALID
