"""Gradients of the combine and of the dispatch on the GPU against their definitions in 64 bits.

Tolerances.  A bf16 result is off by half a step, 2^-8 of its value, an fp32 one by 2^-24.  The
dot products of H terms run in strands of 32 a pass over 8192 columns, with a tree of at most 13
sums above them: each term is rounded at most 48 times up to 8192 columns, 80 times up to 16384."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _inputs(T, H, K, dt=F32, drop=0.0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    slot = torch.randperm(T * K, generator=g, device=DEV).to(I32).view(T, K)
    if drop:
        slot[torch.rand(T, K, generator=g, device=DEV) < drop] = -1
    return r(T, H).to(dt), r(T * K, H).to(BF), slot, torch.rand(T, K, generator=g, device=DEV), r(T, H).to(dt)


def _combine(dY, Yp, slot, w, want_dw=True, dYp=None):
    T, K = slot.shape
    dYp = torch.full_like(Yp, 7.0) if dYp is None else dYp
    dw = torch.full((T, K), 7.0, device=DEV) if want_dw else None
    B.moe_combine_backward(dY, Yp if want_dw else None, slot, w, dYp, dw)
    return dYp, dw


def _combine_reference(dY, Yp, slot, w):
    s = slot.long().clamp(min=0)
    live = (slot >= 0)[..., None]
    rows = dY.to(F64)[:, None] * (1.0 if w is None else w.to(F64)[..., None])
    dYp = torch.full(Yp.shape, 7.0, dtype=F64, device=DEV)
    dYp[slot[slot >= 0].long()] = rows.expand(*slot.shape, -1)[slot >= 0]
    terms = dY.to(F64)[:, None] * Yp.to(F64)[s] * live
    return dYp, terms.sum(-1), terms.abs().sum(-1)


SHAPES = [(1, 64, 1), (45, 256, 2), (7, 320, 32), (300, 2112, 3), (33, 7168, 8), (5, 8256, 4), (3, 16384, 2), (20, 8192, 9)]


@pytest.mark.parametrize("T,H,K", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("weighted,drop", [(True, 0.0), (False, 0.3)])
def test_combine(T, H, K, dt, weighted, drop):
    dY, Yp, slot, w, _ = _inputs(T, H, K, dt, drop)
    w = w if weighted else None
    dYp, dw = _combine(dY, Yp, slot, w)
    ref, rdw, size = _combine_reference(dY, Yp, slot, w)
    assert bool(((dYp.to(F64) - ref).abs() <= (HALF[BF] + 2 ** -23) * ref.abs()).all())
    assert bool(((dw.to(F64) - rdw).abs() <= (48 if H <= 8192 else 80) * 2.0 ** -24 * size).all())
    # without the weights' gradient, and over the rows that were read: the same rows
    again, _ = _combine(dY, Yp, slot, w, want_dw=False)
    assert torch.equal(again, dYp)
    kept = torch.ones(T * K, dtype=torch.bool, device=DEV)
    kept[slot[slot >= 0].long()] = False
    over = Yp.clone()
    _, dw2 = _combine(dY, over, slot, w, dYp=over)
    assert torch.equal(dw2, dw) and torch.equal(over[~kept], dYp[~kept]) and torch.equal(over[kept], Yp[kept])


@pytest.mark.parametrize("T,H,K", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_res,drop", [(True, 0.3), (False, 0.0)])
def test_dispatch(T, H, K, dt, with_res, drop):
    _, rows, slot, _, res = _inputs(T, H, K, dt, drop)
    res = res if with_res else None
    dX = torch.full((T, H), 7.0, device=DEV).to(dt)
    B.moe_dispatch_backward(rows, slot, res, dX)
    terms = rows.to(F64)[slot.long().clamp(min=0)] * (slot >= 0)[..., None]
    ref, size = terms.sum(1), terms.abs().sum(1)
    if with_res:
        ref, size = ref + res.to(F64), size + res.to(F64).abs()
    assert bool(((dX.to(F64) - ref).abs() <= HALF[dt] * ref.abs() + (K + 1) * 2.0 ** -23 * size).all())
    if with_res:                                # added into its own memory
        B.moe_dispatch_backward(rows, slot, res, res)
        assert torch.equal(res, dX)


def test_indices_outside_contribute_nothing_and_rows_without_a_pair_are_not_read():
    T, H, K = 6, 192, 3
    dY, Yp, slot, w, _ = _inputs(T, H, K)
    free = slot[2].long().clone()
    Yp[free] = float("nan")
    slot[2] = torch.tensor([-1, T * K, 2 ** 31 - 1], dtype=I32, device=DEV)
    dYp, dw = _combine(dY, Yp, slot, w)
    assert float(dw[2].abs().max()) == 0.0 and bool(torch.isfinite(dw).all())
    assert bool((dYp[free] == 7.0).all())
    dX = torch.full((T, H), 7.0, device=DEV)
    B.moe_dispatch_backward(Yp, slot, None, dX)
    assert float(dX[2].abs().max()) == 0.0 and bool(torch.isfinite(dX).all())


def test_against_differences_of_the_forward_pass():
    # <d, J v> for the library's own forward calls: Y is linear in Yp and in the weights
    T, H, E, K = 64, 256, 16, 2
    dY, _, _, w, _ = _inputs(T, H, K)
    g = torch.Generator(device=DEV).manual_seed(3)
    X = torch.randn(T, H, generator=g, device=DEV).to(BF)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, 1).indices.to(I32)
    counts, off = torch.empty(E, dtype=I32, device=DEV), torch.empty(E + 1, dtype=I32, device=DEV)
    perm, slot = torch.empty(T * K, dtype=I32, device=DEV), torch.empty(T, K, dtype=I32, device=DEV)
    Xp = torch.empty(T * K, H, dtype=BF, device=DEV)
    ws = torch.zeros(B.moe_workspace_bytes(T, H, E, K, 64, 0), dtype=torch.uint8, device=DEV)
    B.moe_dispatch(X, idx, E, counts, off, perm, slot, Xp, None, ws)

    def combine(rows, weights):
        Y = torch.empty(T, H, device=DEV)
        B.moe_combine(rows, slot, weights, None, Y)
        return Y.to(F64)
    dYp, dw = _combine(dY, Xp, slot, w)
    dX = torch.empty(T, H, device=DEV)
    B.moe_dispatch_backward(dYp, slot, None, dX)
    base = combine(Xp, w)
    v = torch.randn(T, H, generator=g, device=DEV).to(BF)           # a step of the tokens' rows
    vp = v[perm.long()]
    lhs = (dY.to(F64) * combine(vp, w)).sum()
    size = float((dY.to(F64).abs() * combine(vp.abs(), w)).sum())
    assert abs(float(lhs - (dX.to(F64) * v.to(F64)).sum())) <= (2.0 ** -8 + 2.0 ** -16) * size
    u = torch.rand(T, K, generator=g, device=DEV)                   # a step of the weights
    lhs = (dY.to(F64) * (combine(Xp, w + u) - base)).sum()
    size = float((dY.to(F64).abs() * combine(Xp.abs(), w + u)).sum())
    assert abs(float(lhs - (dw.to(F64) * u.to(F64)).sum())) <= 2.0 ** -16 * size


def test_long_arrays_other_stream_and_graph():
    # more than 2^32 bytes and 2^31 elements of rows
    T, H, K = 70000, 4096, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    Yp = torch.empty(T * K, H, dtype=BF, device=DEV).normal_(generator=g)
    slot = torch.randperm(T * K, generator=g, device=DEV).to(I32).view(T, K)
    dY, w = torch.randn(T, H, generator=g, device=DEV), torch.rand(T, K, generator=g, device=DEV)
    dYp, dw, dX = torch.empty_like(Yp), torch.empty(T, K, device=DEV), torch.empty(T, H, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_combine_backward(dY, Yp, slot, w, dYp, dw, stream=side)
    B.moe_dispatch_backward(dYp, slot, None, dX, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for t in (0, 1, T // 2, T - 2, T - 1):
        at = slot[t].long()
        rows = dY[t].to(F64) * w[t].to(F64)[:, None]
        assert bool(((dYp[at].to(F64) - rows).abs() <= (HALF[BF] + 2 ** -23) * rows.abs()).all())
        terms = Yp[at].to(F64) * dY[t].to(F64)
        assert bool(((dw[t].to(F64) - terms.sum(1)).abs() <= 48 * 2.0 ** -24 * terms.abs().sum(1)).all())
        ref = dYp[at].to(F64)
        assert bool(((dX[t].to(F64) - ref.sum(0)).abs() <= 9 * 2.0 ** -24 * ref.abs().sum(0)).all())
    graph = torch.cuda.CUDAGraph()
    want = dYp[:1000].clone(), dw.clone(), dX.clone()
    with torch.cuda.graph(graph):
        B.moe_combine_backward(dY, Yp, slot, w, dYp, dw)
        B.moe_dispatch_backward(dYp, slot, None, dX)
    dYp.zero_(), dw.zero_(), dX.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dYp[:1000], want[0]) and torch.equal(dw, want[1]) and torch.equal(dX, want[2])
