"""Orthogonalised updates on the GPU with few rows or columns, where roundings do not average out: what is off
before the result's own rounding.

That rounding is averaged away: `out` is called for with N scales s = 2^(j / N), and out / s averaged.  A
rounding to bf16 is off by at most 2^-8 of a value, evenly, so at most 2^-8 / sqrt(3) in the mean square; the N
roundings of an entry fall on different places between neighbours, so the mean is 2^-8 / sqrt(3 N) off, in a
2-norm over k entries up to (1 + 5 / sqrt(k)) times that (five standard deviations).

Up to 64 on the smaller side every operand is two fp16 numbers, 22 bits: an entry is off by at most 2^-22, 2^-22 /
sqrt(3) in the mean square.  With |X|_2 <= 1.2 and the default coefficients the products b A X + c A A X carry
that with at most 6.9 + 4.2 = 11.1, for X, for A twice and for P: sqrt(1 + 4 + 1) in the mean square, 3.8e-6 |X|_F a
step.  What of it lies in directions that X lacks grows by a = 3.44 in every step that follows: 141, 41, 12, 3.4
and 1 times, 147 in the mean square: FEW = 147 * 3.8e-6 = 5.6e-4."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FEW = 5.6e-4
KINDS = ["flat", "fall", "low", "one"]


def _matrices(Bn, R, C, kind, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    k = min(R, C)
    if kind == "flat":
        return r(Bn, R, C)
    if kind in ("low", "one"):                  # rank far below the sides
        q = max(1, k // 16) if kind == "low" else 1
        return r(Bn, R, q) @ r(Bn, q, C)
    fall = torch.arange(1, k + 1, device=DEV, dtype=F32) ** -1.0
    return (r(Bn, R, k) * fall) @ r(Bn, k, C) + 0.01 * r(Bn, R, C)


def _reference(u, steps=5):
    u = u.to(F64)
    x = u.mT if u.shape[1] > u.shape[2] else u
    n = torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    x = x / torch.where(n > 0, n, torch.ones_like(n))
    for _ in range(steps):
        A = x @ x.mT
        x = 3.4445 * x + (-4.7750 * A + 2.0315 * (A @ A)) @ x
    return x.mT if u.shape[1] > u.shape[2] else x


def _workspace(shape, fill=0):
    ws = torch.full((B.moe_orthogonalize_workspace_bytes(*shape),), fill, dtype=torch.uint8, device=DEV)
    ws[:256] = 0
    return ws


def _off_before_rounding(g, ref, N=64):
    """-> 2-norms relative to the matrices', and what the mean of the roundings may have left in them"""
    ws, out = _workspace(g.shape), torch.empty(g.shape, device=DEV, dtype=BF)
    mean = torch.zeros(g.shape, device=DEV, dtype=F64)
    for j in range(N):
        s = torch.tensor(2.0 ** (j / N), dtype=F32).item()
        B.moe_orthogonalize(g, out, ws, scale=s)
        mean += out.to(F64) / s
    assert B.moe_read_status(ws) == 0
    d = torch.linalg.vector_norm(mean / N - ref, dim=(1, 2)) / torch.linalg.vector_norm(ref, dim=(1, 2))
    k = g.shape[1] * g.shape[2]
    return float(d.max()), 2.0 ** -8 / (3 * N) ** 0.5 * (1 + 5 / k ** 0.5)


# one CTA a matrix, and clusters of two, four and eight
SHAPES = [(64, 1, 1), (64, 1, 40), (64, 2, 2), (64, 4, 4), (64, 8, 8), (64, 5, 3), (64, 16, 16), (64, 40, 40), (64, 64, 64),
          (64, 63, 65), (64, 200, 33), (64, 384, 64), (64, 64, 128), (64, 2, 385), (64, 32, 500), (64, 64, 768), (64, 777, 17),
          (64, 1500, 4), (64, 64, 1531), (64, 4, 3000), (64, 32, 3000), (64, 3000, 8), (64, 57, 3001), (64, 64, 2500)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_few_rows_or_columns(shape, kind):
    g = _matrices(*shape, kind)
    off, left = _off_before_rounding(g, _reference(g))
    assert off <= FEW + left


# One shape to a launch over a list of tiles: A and P in two numbers, X in one for the products.  Its rounding, 2^-11
# an entry and 2^-11 / sqrt(3) in the mean square, enters each product with P once and A in two places, over sums of
# n > 3000 entries that average it out; so a step adds |P - a I| <= 11.1 times it at most where it does not
# average, 3.1e-3 |X|_F, and five steps of random roundings sqrt(5) of that where all singular values lie at
# |P - a I|'s largest, s = 1.2.  They lie around 1, where |P - a I| = 2.7: THIN = 2.7 * 2^-11 / sqrt(3) * sqrt(5) = 1.7e-3.
THIN = 1.7e-3


@pytest.mark.parametrize("shape", [(64, 1, 3100), (64, 2, 3100), (64, 4, 4096), (64, 8, 5000), (64, 3201, 16), (64, 32, 3300), (64, 4096, 33),
                                   (16, 64, 5000), (2, 7168, 24), (1, 16, 7168), (3, 64, 7169), (30, 7168, 64), (2, 32768, 8), (1, 3, 32768)])
@pytest.mark.parametrize("kind", KINDS)
def test_few_rows_or_columns_of_great_length(shape, kind):
    g = _matrices(*shape, kind)
    off, left = _off_before_rounding(g, _reference(g))
    assert off <= THIN + left


@pytest.mark.parametrize("shape", [(200, 1, 3100), (200, 4843, 1), (200, 2, 4000), (1, 24, 32768)])
def test_few_mantissas_of_great_length(shape):
    for kind in ("fall", "one"):
        g = _matrices(*shape, kind).to(BF)
        off, left = _off_before_rounding(g, _reference(g))
        assert off <= THIN + left


@pytest.mark.parametrize("shape", [(2, 4, 4096), (1, 7168, 24), (200, 64, 4000), (3, 3333, 63)])
def test_great_length_repeats_in_a_graph_and_records_waits(shape):
    g, ws = _matrices(*shape, "fall").to(BF), _workspace(shape, 255)
    out, again = (torch.empty(shape, device=DEV, dtype=BF) for _ in range(2))
    B.moe_orthogonalize(g, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_orthogonalize(g, again, ws)
    for _ in range(3):
        again.zero_()
        graph.replay()
        assert torch.equal(again, out)
    assert B.moe_read_status(ws) == 0
    B.moe_debug_set_wait_limit(2_000_000, 1)
    try:
        B.moe_orthogonalize(g, again, ws)
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    B.moe_orthogonalize(g, again, ws)
    assert B.moe_read_status(ws) == 0 and torch.equal(again, out)


@pytest.mark.parametrize("shape", [(5, 24, 40), (5, 300, 64), (5, 30, 700), (5, 2900, 9), (5, 6, 3200)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_momentum_steps_zeros_and_nan_with_few_rows(shape, dt):
    g, m = _matrices(*shape, "flat").to(dt), _matrices(*shape, "fall", seed=1)
    g[1], m[1] = 0.0, 0.0
    g[2, 0, 0] = float("nan")
    g[3, 1, 2] = float("inf")
    u = g.to(F64) + 0.9 * (0.9 * m.to(F64) + g.to(F64))
    for steps in (1, 2, 5):
        ws, out, mo = _workspace(shape), torch.full(shape, 7.0, device=DEV, dtype=BF), m.clone()
        B.moe_orthogonalize(g, out, ws, momentum=mo, mu=0.9, nesterov=True, steps=steps)
        assert B.moe_read_status(ws) == 0 and float(out[1].abs().max()) == 0.0
        assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())
        for i in (0, 4):
            ref = _reference(u[i:i + 1], steps)
            assert float((out[i].to(F64) - ref[0]).norm()) <= (THIN + 2.0 ** -8) * float(ref.norm())


@pytest.mark.parametrize("shape", [(4, 40, 56), (4, 41, 57), (4, 100, 90), (4, 60, 1000), (4, 333, 250), (4, 8, 3200)])
@pytest.mark.parametrize("momentum", [False, True])
def test_subnormal_entries(shape, momentum):
    # (made on the host, so that nothing on the way takes them for zero; the reference takes them as they are)
    g = _matrices(*shape, "flat").cpu().to(F64)
    for i, size in enumerate((1e-39, 1e-41, 1e-43, 3e-45)):
        g[i] *= size / float(g[i].abs().max())
    for dt in (F32, BF):
        u = g.to(F32).to(dt)
        live = [i for i in range(4) if float(u[i].to(F64).abs().max()) > 0.0]
        assert live == ([0, 1, 2, 3] if dt == F32 else [0])      # (bf16's smallest number is 9.2e-41)
        ref = _reference(u.to(DEV))
        ws, out = _workspace(shape), torch.full(shape, 7.0, device=DEV, dtype=BF)
        m = torch.zeros(shape, device=DEV) if momentum else None
        B.moe_orthogonalize(u.to(DEV), out, ws, momentum=m)
        assert B.moe_read_status(ws) == 0
        for i in range(4):
            # (sides above 64: the updates' own error; 6.2e-3 bounds it)
            assert float((out[i].to(F64) - ref[i]).norm()) <= (6.2e-3 + 2.0 ** -8) * float(ref[i].norm()), (dt, i)


@pytest.mark.parametrize("shape", [(3, 40, 56), (3, 300, 64), (3, 30, 700), (3, 700, 21), (5, 64, 2999), (2, 6, 3200), (2, 3300, 64)])
def test_few_rows_over_their_own_memory_and_in_graphs(shape):
    g, ws = _matrices(*shape, "fall").to(BF), _workspace(shape, 255)
    out, same = torch.empty_like(g), g.clone()
    B.moe_orthogonalize(g, out, ws)
    B.moe_orthogonalize(same, same, ws)
    assert torch.equal(same, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_orthogonalize(g, same, ws)
    for _ in range(2):
        same.zero_()
        graph.replay()
        assert torch.equal(same, out)
    B.moe_debug_set_wait_limit(2_000_000, 1)
    try:
        B.moe_orthogonalize(g, same, ws)
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    B.moe_orthogonalize(g, same, ws)
    assert B.moe_read_status(ws) == 0 and torch.equal(same, out)


def test_calls_of_every_kind_at_once():
    shapes = [(64, 32, 3000), (200, 40, 40), (30, 700, 60), (40, 128, 1024), (3, 4096, 33), (6, 300, 520)]
    gs = [_matrices(*s, "fall").to(BF) for s in shapes]
    outs, wss, streams = [torch.empty_like(g) for g in gs], [_workspace(s) for s in shapes], [torch.cuda.Stream() for _ in shapes]
    want = [torch.empty_like(g) for g in gs]
    for g, o, ws in zip(gs, want, wss):
        B.moe_orthogonalize(g, o, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, o, ws, st in zip(gs, outs, wss, streams):
            B.moe_orthogonalize(g, o, ws, stream=st)
    torch.cuda.synchronize()
    for o, w, ws in zip(outs, want, wss):
        assert torch.equal(o, w) and B.moe_read_status(ws) == 0
