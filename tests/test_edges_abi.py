"""Argument checks of the entry points at the layer's edges (the combine's and the dispatch's
gradients, the joined residual and its norms): a bad call is refused on the host before anything
reaches a GPU (CPU only: no call here launches a kernel)."""
import ctypes

import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

P = ctypes.c_void_p
OK, BAD, WS = P(0x10000), P(0x10004), P(0x100000)     # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return B.load()


def test_combine_backward_refusals(lib):
    def call(d=OK, f32=1, y=OK, s=OK, w=OK, T=4, H=128, K=2, o=OK, dw=OK):
        return lib.moe_combine_backward(d, f32, y, s, w, T, H, K, o, dw, None)
    assert call(T=-1) == -1 and call(H=0) == -1 and call(K=0) == -1 and call(f32=2) == -1
    assert call(H=96) == -2 and call(K=33) == -2 and call(T=1 << 28, K=8) == -2
    assert call(d=None) == -1 and call(y=None) == -1 and call(s=None) == -1 and call(o=None) == -1
    assert call(d=BAD) == -3 and call(w=BAD) == -3 and call(dw=BAD) == -3 and call(o=BAD) == -3
    assert call(T=0, d=None, y=None, s=None, w=None, o=None, dw=None) == 0


def test_dispatch_backward_refusals(lib):
    def call(d=OK, s=OK, r=None, T=4, H=128, K=2, o=OK, f32=0):
        return lib.moe_dispatch_backward(d, s, r, T, H, K, o, f32, None)
    assert call(T=-1) == -1 and call(H=-64) == -1 and call(K=-1) == -1 and call(f32=-1) == -1
    assert call(H=32) == -2 and call(K=33) == -2
    assert call(d=None) == -1 and call(s=None) == -1 and call(o=None) == -1
    assert call(d=BAD) == -3 and call(s=BAD) == -3 and call(r=BAD) == -3
    assert call(T=0, d=None, s=None, o=None) == 0


def _options(post=1, pre=2, alpha=1.0, eps=1e-5, gp=OK, bp=None, g=None, gt=None, gq=OK, bq=None):
    return B.MoeResidual(post, pre, alpha, eps, eps, gp, bp, g, gt, gq, bq)


def test_residual_refusals(lib):
    def fwd(p=None, x=OK, xf=1, y=OK, yf=0, T=4, H=128, r=OK, n=OK, st=None):
        p = _options() if p is None else p
        return lib.moe_residual_norm(x, xf, y, yf, ctypes.byref(p), T, H, r, n, st, None)

    def bwd(p=None, dn=OK, dr=OK, y=OK, yf=0, r=OK, xf=1, st=OK, T=4, H=128, dx=OK, dy=OK, g=None, ws=WS, n=BIG):
        p = _options() if p is None else p
        return lib.moe_residual_norm_backward(dn, dr, y, yf, r, xf, st, ctypes.byref(p), T, H, dx, dy,
                                              None if g is None else ctypes.byref(g), ws, n, None)
    for f in (fwd, bwd):
        assert f(T=-1) == -1 and f(H=0) == -1 and f(xf=2) == -1 and f(yf=-1) == -1
        assert f(H=100) == -2 and f(H=16448) == -2 and f(T=0x7fffffff) == -2
        assert f(p=_options(post=3)) == -1 and f(p=_options(pre=-1)) == -1
        assert f(p=_options(alpha=float("nan"))) == -1
        assert f(p=_options(eps=-1.0)) == -1 and f(p=_options(eps=float("nan"))) == -1
        assert f(p=_options(gp=None)) == -1 and f(p=_options(gq=None)) == -1
        assert f(p=_options(bp=BAD)) == -3 and f(p=_options(bq=BAD)) == -3
        assert f(p=_options(g=BAD)) == -3 and f(p=_options(gt=BAD)) == -3
        assert f(y=None) == -1
    assert fwd(x=None) == -1 and fwd(r=None) == -1 and fwd(n=None) == -1 and fwd(st=BAD) == -3
    assert fwd(T=0, x=None, y=None, r=None, n=None) == 0
    assert lib.moe_residual_norm(OK, 1, OK, 1, None, 4, 128, OK, OK, None, None) == -1
    assert bwd(dn=None) == -1 and bwd(r=None) == -1 and bwd(st=None) == -1 and bwd(dx=None) == -1 and bwd(dy=None) == -1
    assert bwd(ws=None) == -1 and bwd(ws=P(0x100010)) == -3 and bwd(dr=BAD) == -3
    # without the next norm, the stream's gradient has to come from dr
    assert bwd(p=_options(pre=0), dr=None) == -1
    # gradients of parameters that the call does not have
    for k in range(6):
        g = B.MoeResidualGrads(*[OK if i == k else None for i in range(6)])
        assert bwd(p=_options(post=0, pre=0, gp=None, gq=None), g=g) == -1
    assert bwd(g=B.MoeResidualGrads(BAD, None, None, None, None, None)) == -3
    need = B.moe_residual_norm_backward_workspace_bytes(4, 128)
    assert need > 0 and bwd(n=need - 1) == -4
    assert B.moe_residual_norm_backward_workspace_bytes(4, 100) == 0
    assert B.moe_residual_norm_backward_workspace_bytes(-1, 128) == 0


def test_bindings_check_types_and_sizes():
    t = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype)
    bf, i32 = torch.bfloat16, torch.int32
    with pytest.raises(ValueError, match="dY"):
        B.moe_combine_backward(t(4, 64, dtype=torch.float16), t(8, 64, dtype=bf), t(4, 2, dtype=i32), t(4, 2), t(8, 64, dtype=bf))
    with pytest.raises(ValueError, match="dYp: 256 elements"):
        B.moe_combine_backward(t(4, 64), t(8, 64, dtype=bf), t(4, 2, dtype=i32), t(4, 2), t(4, 64, dtype=bf))
    with pytest.raises(ValueError, match="dres: dtype"):
        B.moe_dispatch_backward(t(8, 64, dtype=bf), t(4, 2, dtype=i32), t(4, 64), t(4, 64, dtype=bf))
    with pytest.raises(ValueError, match="gamma_pre: 32 elements"):
        B.moe_residual_norm(t(4, 64), t(4, 64), dict(pre="rms", gamma_pre=t(32)), t(4, 64))
    with pytest.raises(ValueError, match="gamma: unknown"):
        B.moe_residual_norm(t(4, 64), t(4, 64), dict(gamma=t(64)), t(4, 64))
    with pytest.raises(ValueError, match="pre: group"):
        B.moe_residual_norm(t(4, 64), t(4, 64), dict(pre="group"), t(4, 64))


def test_orthogonalize_refusals(lib):
    def call(g=OK, f32=0, m=None, mu=0.95, nesterov=0, Bn=2, R=64, C=96, steps=5, co=None, scale=1.0, o=OK, ws=WS, n=BIG):
        return lib.moe_orthogonalize(g, f32, m, mu, nesterov, Bn, R, C, steps, co, scale, o, ws, n, None)
    nan = float("nan")
    assert call(Bn=-1) == -1 and call(R=0) == -1 and call(C=-3) == -1 and call(f32=2) == -1 and call(nesterov=2, m=OK) == -1
    assert call(steps=0) == -1 and call(nesterov=1) == -1 and call(mu=nan) == -1 and call(scale=nan) == -1
    assert call(steps=33) == -2 and call(R=32769) == -2 and call(C=32769) == -2 and call(Bn=65536) == -2
    assert call(co=ctypes.cast((ctypes.c_float * 15)(*[1.0] * 14, nan), P)) == -1
    assert call(g=None) == -1 and call(o=None) == -1 and call(ws=None) == -1
    assert call(g=BAD) == -3 and call(m=BAD) == -3 and call(o=BAD) == -3 and call(ws=P(0x100010)) == -3
    need = B.moe_orthogonalize_workspace_bytes(2, 64, 96)
    assert need > 0 and call(n=need - 1) == -4
    assert call(Bn=0, g=None, o=None, ws=None) == 0
    assert B.moe_orthogonalize_workspace_bytes(1, 0, 4) == 0 and B.moe_orthogonalize_workspace_bytes(1, 4, 32769) == 0
    t = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype)
    with pytest.raises(ValueError, match="out: dtype"):
        B.moe_orthogonalize(t(4, 8), t(4, 8), t(256))
    with pytest.raises(ValueError, match="momentum: 16 elements"):
        B.moe_orthogonalize(t(4, 8), t(4, 8, dtype=torch.bfloat16), t(256), momentum=t(16))
    with pytest.raises(ValueError, match="coeffs: 3 values, expected 6"):
        B.moe_orthogonalize(t(4, 8), t(4, 8, dtype=torch.bfloat16), t(256), steps=2, coeffs=[(1, 2, 3)])


def test_rows_longer_than_the_grid_are_refused(lib):
    assert lib.moe_combine_backward(OK, 0, OK, OK, OK, 1, (1 << 25) + 64, 1, OK, OK, None) == -2
    assert lib.moe_dispatch_backward(OK, OK, None, 1, (1 << 26) + 64, 1, OK, 0, None) == -2
