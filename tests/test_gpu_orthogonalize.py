"""Orthogonalised updates on the GPU against the definition in 64 bits.

Tolerances.  The bf16 result is off by half a step, 2^-8 of its value.  Before that, every step
rounds the operands X, A and P of its products to fp16, 2^-11 of each entry at most and 2^-11 /
sqrt(3) in the mean square.  With |X|_2 <= 1.2 and the default coefficients, the products P X = b A X +
c A A X (a X is carried in more bits; with a I in P the sum is smaller, not larger: they cancel) carry
these with |b| |X|^2 + |c| |X|^4 <= 6.9 + 4.2 at most, twice for A (two factors), so a step adds at most
(6.9 + 4.2) * (1 + 2 + 1) * 2^-11 / sqrt(3) = 1.25e-2 |X|_F in the worst alignment of five steps' errors.  They are independent and most of them act where the factors are far below their
bounds; a direction's own error is divided by its size, and |p'| < 1 near the fixed points.  NEAR is
half of one such worst step; what is held against the formula in 2-norm is below a third of it
(measured on the CPU with the same roundings: 0.3e-3 to 1.8e-3 over flat, falling and low-rank
spectra)."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ABC = (3.4445, -4.7750, 2.0315)
NEAR = 6.2e-3


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _matrices(Bn, R, C, kind="fall", seed=0):
    g = _gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    k = min(R, C)
    if kind == "flat":
        return r(Bn, R, C)
    if kind == "low":                           # rank far below the sides
        q = max(1, k // 16)
        return r(Bn, R, q) @ r(Bn, q, C)
    fall = torch.arange(1, k + 1, device=DEV, dtype=F32) ** -1.0
    return (r(Bn, R, k) * fall) @ r(Bn, k, C) + 0.01 * r(Bn, R, C)


def _reference(u, steps=5, coeffs=None, scale=1.0):
    u = u.to(F64)
    x = u.mT if u.shape[1] > u.shape[2] else u
    n = torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    x = x / torch.where(n > 0, n, torch.ones_like(n))
    for k in range(steps):
        a, b, c = ABC if coeffs is None else coeffs[k]
        A = x @ x.mT
        x = a * x + (b * A + c * (A @ A)) @ x
    return scale * (x.mT if u.shape[1] > u.shape[2] else x)


def _run(g, stream=None, out=None, ws=None, **kw):
    Bn, R, C = g.shape
    out = torch.full(g.shape, 7.0, device=DEV, dtype=BF) if out is None else out
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(Bn, R, C), dtype=torch.uint8, device=DEV) if ws is None else ws
    B.moe_orthogonalize(g, out, ws, stream=stream, **kw)
    assert stream is not None or torch.cuda.is_current_stream_capturing() or B.moe_read_status(ws) == 0
    return out


def _off(got, ref):
    """Largest relative 2-norm over the matrices"""
    d = torch.linalg.vector_norm(got.to(F64) - ref, dim=(1, 2))
    return float((d / torch.linalg.vector_norm(ref, dim=(1, 2)).clamp(min=1e-300)).max())


SHAPES = [(1, 1, 1), (3, 1, 40), (2, 40, 1), (2, 7, 9), (3, 33, 65), (4, 64, 64), (5, 129, 100), (2, 128, 256), (16, 256, 128),
          (1, 255, 257), (2, 257, 255), (3, 300, 520), (1, 1088, 2112), (2, 2112, 1088), (1, 1000, 1001), (2, 600, 130),
          (1, 16, 7168), (1, 7168, 24), (700, 24, 17), (40, 192, 320), (2, 128, 384), (3, 383, 128), (2, 128, 392), (1, 136, 384),
          (2, 96, 264), (2, 64, 321), (2, 1, 1000), (1, 1000, 1), (3, 5, 385), (2, 768, 128), (2, 128, 769), (3, 1537, 100),
          (2, 77, 1531), (40, 128, 1024), (1, 128, 3000), (2, 3001, 57), (1, 120, 3090), (2, 129, 1500)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["flat", "fall", "low"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_against_the_definition(shape, kind, dt):
    g = _matrices(*shape, kind).to(dt)
    out = _run(g)
    ref = _reference(g)
    assert _off(out, ref) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    size = ref.square().mean((1, 2), keepdim=True).sqrt()
    assert bool(((out.to(F64) - ref).abs() <= 2.0 ** -8 * ref.abs() + 8 * NEAR * torch.maximum(size, ref.abs())).all())


def test_full_width():
    for shape in ((2, 7168, 2048), (1, 2048, 7168)):
        g = _matrices(*shape, "fall").to(BF)
        assert _off(_run(g), _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5


@pytest.mark.parametrize("shape", [(3, 33, 65), (2, 256, 128), (2, 264, 136), (2, 1001, 65), (2, 128, 800)])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_momentum(shape, nesterov, dt):
    g, m = _matrices(*shape, "flat").to(dt), 3 * _matrices(*shape, "fall", seed=1)
    want = 0.9 * m.to(F64) + g.to(F64)
    u = g.to(F64) + 0.9 * want if nesterov else want
    kept = m.clone()
    out = _run(g, momentum=m, mu=0.9, nesterov=nesterov)
    # mu is 0.9 rounded to fp32; one rounding of the fused product and sum
    assert bool(((m.to(F64) - want).abs() <= 2.0 ** -24 * (want.abs() + kept.abs().to(F64))).all())
    assert _off(out, _reference(u)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5


def test_coefficients_scale_steps_and_own_memory():
    g = _matrices(2, 96, 160, "flat").to(BF)
    co = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    out = _run(g, steps=3, coeffs=co, scale=0.2)
    ref = _reference(g, 3, co, 0.2)
    assert _off(out, ref) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    same = g.clone()
    assert torch.equal(_run(same, steps=3, coeffs=co, scale=0.2, out=same), out)
    g = _matrices(2, 300, 200, "flat").to(BF)
    same = g.clone()
    assert torch.equal(_run(same, out=same), _run(g))
    for steps in (1, 2):                        # (the last and the last but one carry X in fewer numbers)
        assert _off(_run(g, steps=steps), _reference(g, steps)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    g = g[:, :96].contiguous()
    assert _off(_run(g, steps=1), _reference(g, 1)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5


@pytest.mark.parametrize("shape", [(6, 40, 56), (6, 41, 57), (6, 60, 1000), (6, 333, 250)])
def test_sizes_zeros_infinities_and_nan(shape):
    g = _matrices(*shape, "flat")
    ref = _reference(g)
    g[0] *= 1e-36
    g[1] *= 2.0 ** 124 / float(g[1].abs().max())
    g[2] = 0.0
    g[3, 2, 3] = float("inf")
    g[4, 5, 6] = float("nan")
    out = _run(g)
    # (1e-36 itself rounds the entries to normal fp32 numbers)
    for i in (0, 1, 5):
        assert _off(out[i:i + 1], ref[i:i + 1]) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    assert float(out[2].abs().max()) == 0.0
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[4]).all())


@pytest.mark.parametrize("shape", [(5, 300, 520), (5, 521, 303), (5, 100, 200)])
@pytest.mark.parametrize("momentum", [False, True])
def test_uneven_matrices(shape, momentum):
    # entries that a sample of the matrix says little of: one row, one entry, columns and rows whose sizes
    # fall off over many powers of ten, a single large entry among others
    _, R, C = shape
    g = _matrices(*shape, "flat")
    row, entry = g[0, 7].clone(), g[1, 3, 4].clone()
    g[0], g[1] = 0.0, 0.0
    g[0, 7], g[1, 3, 4] = row, entry
    g[2] *= 10.0 ** (-torch.arange(C, device=DEV) / (C / 8))
    g[3] *= 10.0 ** (-torch.arange(R, device=DEV) / (R / 8))[:, None]
    g[4, 5, 9] = 1e4
    m = torch.zeros_like(g) if momentum else None
    out = _run(g, momentum=m, nesterov=momentum)
    assert _off(out, _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    assert m is None or torch.equal(m, g)


def test_repeats_and_batches_bit_for_bit():
    g = _matrices(5, 300, 200, "fall").to(BF)
    out = _run(g)
    assert torch.equal(_run(g), out)
    for i in range(5):
        assert torch.equal(_run(g[i:i + 1].contiguous())[0], out[i])
    flat = torch.empty(300, 200, dtype=BF, device=DEV)
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(1, 300, 200), dtype=torch.uint8, device=DEV)
    B.moe_orthogonalize(g[0].contiguous(), flat, ws)
    assert torch.equal(flat, out[0])


# (few matrices with long sums: A = X X^T in parts that the last one adds)
LONG = [(1, 7168, 100), (4, 100, 7168), (1, 5001, 300), (6, 200, 2100), (1, 257, 4100), (1, 7168, 24), (2, 1024, 4096), (30, 7168, 64)]


@pytest.mark.parametrize("shape", LONG)
@pytest.mark.parametrize("kind", ["flat", "low"])
def test_long_sums_of_few_matrices(shape, kind):
    g = _matrices(*shape, kind).to(BF)
    ws = torch.full((B.moe_orthogonalize_workspace_bytes(*shape),), 255, dtype=torch.uint8, device=DEV)
    ws[:256] = 0                                # (the status word; the rest is the call's own)
    out = _run(g, ws=ws)
    assert _off(out, _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    for _ in range(3):                          # whichever part comes last
        assert torch.equal(_run(g, ws=ws), out)
    graph, again = torch.cuda.CUDAGraph(), torch.empty_like(out)
    with torch.cuda.graph(graph):
        _run(g, out=again, ws=ws)
    for _ in range(2):
        again.zero_()
        graph.replay()
        assert torch.equal(again, out)


@pytest.mark.parametrize("shape", [(40, 1100, 1024), (2, 1023, 1024), (2, 1024, 1024), (3, 1025, 1100)])
def test_groups_of_matrices_and_both_rings(shape):
    g = _matrices(*shape, "fall").to(BF)
    out = _run(g)
    assert _off(out, _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
    assert torch.equal(_run(g), out)


def test_two_calls_at_once():
    shapes = [(1, 7168, 100), (2, 600, 2100)]
    gs = [_matrices(*s, "fall").to(BF) for s in shapes]
    want = [_run(g) for g in gs]
    wss = [torch.zeros(B.moe_orthogonalize_workspace_bytes(*s), dtype=torch.uint8, device=DEV) for s in shapes]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, o, ws, st in zip(gs, outs, wss, streams):
            _run(g, stream=st, out=o, ws=ws)
    torch.cuda.synchronize()
    for o, w, ws in zip(outs, want, wss):
        assert torch.equal(o, w) and B.moe_read_status(ws) == 0


def test_a_wait_that_runs_out_with_sums_in_parts():
    g = _matrices(1, 7168, 100).to(BF)
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(1, 7168, 100), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(g)
    B.moe_debug_set_wait_limit(2_000_000, 1)
    try:
        B.moe_orthogonalize(g, out, ws)
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    assert _off(_run(g, ws=ws), _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5


def test_other_stream_and_graph():
    g, m0 = _matrices(3, 130, 70, "fall"), _matrices(3, 130, 70, "flat", seed=2)
    m = m0.clone()
    want = _run(g, momentum=m)
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(3, 130, 70), dtype=torch.uint8, device=DEV)
    out, m1 = torch.empty_like(want), m0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _run(g, stream=side, out=out, ws=ws, momentum=m1)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(m1, m)
    m1.copy_(m0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(g, out=out, ws=ws, momentum=m1)
    for _ in range(2):
        m1.copy_(m0)
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(m1, m)
    assert B.moe_read_status(ws) == 0


@pytest.mark.parametrize("shape", [(2, 128, 256), (2, 2500, 96), (2, 300, 200)])
def test_a_wait_that_runs_out_is_recorded(shape):
    g = _matrices(*shape).to(BF)
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(*shape), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(g)
    B.moe_debug_set_wait_limit(2_000_000, 1)
    try:
        B.moe_orthogonalize(g, out, ws)
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    assert _off(_run(g, ws=ws), _reference(g)) <= (NEAR ** 2 + 2.0 ** -16) ** 0.5
