"""Argument checks of the training entry points: a bad call is refused on the host before
anything reaches a GPU (CPU only: no call here launches a kernel)."""
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


def test_layer_norm_refusals(lib):
    f = lib.moe_layer_norm

    def call(x=OK, f32=0, g=OK, b=None, T=4, H=128, eps=1e-5, y=OK, m=None, r=None):
        return f(x, f32, g, b, T, H, eps, y, m, r, None)
    assert call(T=-1) == -1 and call(H=0) == -1 and call(f32=2) == -1
    assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1
    assert call(H=96) == -2 and call(H=16448) == -2
    assert call(x=None) == -1 and call(g=None) == -1 and call(y=None) == -1
    assert call(x=BAD) == -3 and call(b=BAD) == -3 and call(m=BAD) == -3 and call(r=BAD) == -3
    assert call(T=0, x=None, y=None) == 0


def test_layer_norm_backward_refusals(lib):
    f = lib.moe_layer_norm_backward

    def call(dy=OK, x=OK, f32=0, res=None, T=4, H=128, dx=OK, dg=OK, ws=WS, n=BIG):
        return f(dy, x, f32, OK, OK, OK, res, T, H, dx, dg, OK, ws, n, None)
    assert call(T=-1) == -1 and call(f32=-1) == -1 and call(H=100) == -2
    assert call(dy=None) == -1 and call(dx=None) == -1 and call(dg=None) == -1 and call(ws=None) == -1
    assert call(res=BAD) == -3 and call(x=BAD) == -3 and call(ws=P(0x100010)) == -3
    need = B.moe_layer_norm_backward_workspace_bytes(4, 128)
    assert need > 0 and call(n=need - 1) == -4
    assert B.moe_layer_norm_backward_workspace_bytes(4, 100) == 0
    assert B.moe_layer_norm_backward_workspace_bytes(-1, 128) == 0


def test_route_refusals(lib):
    def fwd(l=OK, f32=1, b=None, T=4, E=16, K=2, i=OK, w=OK, r=None):
        return lib.moe_route_logits(l, f32, b, T, E, K, None if r is None else ctypes.byref(r), i, w, None)

    def bwd(l=OK, f32=1, T=4, E=16, K=2, i=OK, w=OK, d=OK, r=None):
        return lib.moe_route_logits_backward(l, f32, T, E, K, None if r is None else ctypes.byref(r), i, w, d, None)
    for f in (fwd, bwd):
        assert f(T=-1) == -1 and f(K=0) == -1 and f(K=17) == -1 and f(f32=3) == -1
        assert f(E=1025) == -2 and f(E=64, K=33) == -2
        assert f(l=None) == -1 and f(i=None) == -1 and f(w=None) == -1 and f(l=BAD) == -3
        assert f(T=0, l=None, i=None, w=None) == 0
        assert f(r=B.MoeRouting(2, 1, 1, 1, 1)) == -1
        assert f(r=B.MoeRouting.make(n_group=3)) == -1
        assert f(r=B.MoeRouting.make(n_group=4, topk_group=2), K=9) == -1
        assert f(E=128, r=B.MoeRouting.make(n_group=64, topk_group=2)) == -2
    assert fwd(b=BAD) == -3 and bwd(d=None) == -1


def test_checkpoint_refusals(lib):
    def unpack(x, rows, n, q, sc, st):
        return lib.moe_checkpoint_unpack(q, sc, rows, n, x, st)
    for f in (lib.moe_checkpoint_pack, unpack):
        assert f(OK, -1, 128, OK, OK, None) == -1 and f(OK, 4, 0, OK, OK, None) == -1
        assert f(OK, 4, 96, OK, OK, None) == -2 and f(OK, 1 << 31, 128, OK, OK, None) == -2
        assert f(OK, 1 << 30, 192, OK, OK, None) == -2          # blocks past 2^31
        assert f(None, 4, 128, OK, OK, None) == -1 and f(OK, 4, 128, OK, BAD, None) == -3
        assert f(None, 0, 128, None, None, None) == 0


def test_binding_checks_types_and_sizes():
    T, H, E, K = 4, 128, 8, 2
    x, y = torch.zeros(T, H), torch.zeros(T, H, dtype=torch.bfloat16)
    g, s = torch.ones(H), torch.zeros(T)
    with pytest.raises(ValueError, match="x: dtype"):
        B.moe_layer_norm(x.double(), g, None, 1e-5, y)
    with pytest.raises(ValueError, match="gamma: 64 elements, expected 128"):
        B.moe_layer_norm(x, g[:64], None, 1e-5, y)
    with pytest.raises(ValueError, match="y: dtype"):
        B.moe_layer_norm(x, g, None, 1e-5, x)
    with pytest.raises(ValueError, match="dres: dtype"):
        B.moe_layer_norm_backward(y, x, g, s, s, y, x, g, g, torch.zeros(8, dtype=torch.uint8))
    l, i, w = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    with pytest.raises(ValueError, match="topk_idx: dtype"):
        B.moe_route_logits(l, None, K, None, i.long(), w)
    with pytest.raises(ValueError, match="bias: 7 elements"):
        B.moe_route_logits(l, torch.zeros(7), K, None, i, w)
    with pytest.raises(ValueError, match="d_logits: dtype"):
        B.moe_route_logits_backward(l, None, i, w, l.bfloat16())
    with pytest.raises(ValueError, match="scale: 4 elements, expected 8"):
        B.moe_checkpoint_pack(torch.zeros(T, 192, dtype=torch.bfloat16), None, torch.zeros(T, 1, dtype=torch.int8))
    with pytest.raises(ValueError, match="device tensors"):
        B.moe_checkpoint_pack(y)


def test_expert_backward_refusals(lib):
    def call(x=OK, xs=None, dY=OK, off=OK, slot=OK, w=OK, T=4, H=128, E=4, K=2, I=64, dX=OK, dw=None, d1=OK,
             ws=WS, n=BIG):
        return lib.moe_expert_ffn_backward(x, xs, dY, off, slot, w, T, H, E, K, I, OK, OK, OK, dX, dw, d1, OK, OK,
                                           ws, n, None)
    assert call(T=-1) == -1 and call(K=5) == -1 and call(I=0) == -1 and call(H=0) == -1
    assert call(H=96) == -2 and call(I=96) == -2 and call(E=1025) == -2 and call(E=64, K=33) == -2
    assert call(T=1 << 30, K=2) == -2
    for name in ("x", "dY", "off", "slot", "dX", "d1", "ws"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "xs", "dY", "off", "slot", "w", "dX", "dw", "d1"):
        assert call(**{name: BAD}) == -3, name
    need = B.moe_expert_ffn_backward_workspace_bytes(4, 128, 4, 2, 64)
    assert call(n=need - 1) == -4 and call(ws=P(0x100080)) == -3
    assert B.moe_expert_ffn_backward_workspace_bytes(4, 100, 4, 2, 64) == 0
    x = torch.zeros(4, 128, dtype=torch.uint8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    W = torch.zeros(4, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: dtype"):       # bytes without their exponents
        B.moe_expert_ffn_backward(x, None, x.bfloat16(), torch.zeros(5, dtype=torch.int32), i, None, W, W, W,
                                  x.bfloat16(), None, W, W, W, x)
    with pytest.raises(ValueError, match="offsets: 4 elements"):
        B.moe_expert_ffn_backward(x.bfloat16(), None, x.bfloat16(), torch.zeros(4, dtype=torch.int32), i, None,
                                  W, W, W, x.bfloat16(), None, W, W, W, x)
