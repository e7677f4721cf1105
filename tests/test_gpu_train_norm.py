"""Layer norm, its backward pass and the 8-bit checkpoint on the GPU against their
definitions in 64 bits.

Tolerances.  A bf16 result is off by half a step, 2^-8 of its value, and an fp32 one by
2^-24, on top of what the fp32 sums before it lose: a sum over n terms in strands of at most
16 with a tree above them rounds each term at most 32 times, so 32 * 2^-24 of the sum of the
terms' magnitudes."""
import numpy as np
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
SUM = 32 * 2.0 ** -24


def _norm_inputs(T, H, xt, seed=0, offset=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = (r(T, H) * (0.2 + 3 * torch.rand(T, 1, generator=g, device=DEV)) + offset).to(xt)
    return x, 1 + 0.2 * r(H), 0.3 * r(H), (0.1 * r(T, H)).to(BF), r(T, H).to(xt)


def _forward(x, gamma, beta, eps=1e-5):
    T, H = x.shape
    y = torch.empty(T, H, dtype=BF, device=DEV)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    B.moe_layer_norm(x, gamma, beta, eps, y, mean, rstd)
    return y, mean, rstd


def _backward(dy, x, gamma, mean, rstd, res, dx=None):
    T, H = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    dg, db = torch.full((H,), 7.0, device=DEV), torch.full((H,), 7.0, device=DEV)
    ws = torch.zeros(B.moe_layer_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    B.moe_layer_norm_backward(dy, x, gamma, mean, rstd, res, dx, dg, db, ws)
    return dx, dg, db


SHAPES = [(1, 64), (3, 256), (45, 320), (17, 512), (9, 960), (33, 1024), (5, 1088), (700, 2112), (130, 7168),
          (2, 8256), (3, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("with_beta", [True, False])
def test_forward(T, H, xt, with_beta):
    x, gamma, beta, _, _ = _norm_inputs(T, H, xt)
    beta = beta if with_beta else None
    y, mean, rstd = _forward(x, gamma, beta)
    X = x.to(F64)
    mu = X.mean(1, keepdim=True)
    r = ((X - mu).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    shift = 0.0 if beta is None else beta.to(F64)
    ref = gamma.to(F64) * (X - mu) * r + shift
    size = X.abs().amax(1, keepdim=True)
    assert bool(((mean.to(F64) - mu[:, 0]).abs() <= SUM * size[:, 0]).all())
    assert bool(((rstd.to(F64) / r[:, 0] - 1).abs() <= 2 * SUM * (1 + size[:, 0] * r[:, 0])).all())
    tol = 2.0 ** -8 * ref.abs() + 4 * SUM * (1 + size * r) * (gamma.to(F64).abs() * size * r + abs(shift))
    assert bool(((y.to(F64) - ref).abs() <= tol).all())


def test_forward_far_from_zero_and_constant_rows():
    # rows around 1000 with unit spread: a sum of squares in fp32 would lose the variance
    x, gamma, beta, _, _ = _norm_inputs(8, 7168, F32, offset=1000.0)
    x[3] = 5.0                                  # no spread: y = beta
    x[4] = 0.0
    y, mean, rstd = _forward(x, gamma, beta)
    X = x.to(F64)
    var = (X - X.mean(1, keepdim=True)).square().mean(1)
    r = (var + 1e-5) ** -0.5
    live = [0, 1, 2, 5, 6, 7]
    # mu is off by SUM * 1000 at most, which moves a spread of >= 0.2 by its square
    assert bool((rstd.to(F64)[live] / r[live] - 1).abs().max() <= 1e-5)
    assert torch.equal(y[4], beta.to(BF)) and bool(torch.isfinite(y).all())
    assert float((y[3].float() - beta).abs().max()) <= 1000 * SUM * 5 / 1e-5 ** 0.5
    assert float(mean[4]) == 0.0 and abs(float(rstd[4]) / 1e-5 ** -0.5 - 1) <= 1e-6


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("with_res", [False, True])
def test_backward(T, H, xt, with_res):
    x, gamma, _, dy, res = _norm_inputs(T, H, xt, seed=1)
    _, mean, rstd = _forward(x, gamma, None)
    dx, dg, db = _backward(dy, x, gamma, mean, rstd, res if with_res else None)
    X, D, G = x.to(F64), dy.to(F64), gamma.to(F64)
    r = rstd.to(F64)[:, None]
    xh = (X - mean.to(F64)[:, None]) * r
    a = G * D
    ref = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    mag = r * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    if with_res:
        ref = ref + res.to(F64)
        mag = mag + res.to(F64).abs()
    step = 2.0 ** -8 if xt == BF else 2.0 ** -24
    assert bool(((dx.to(F64) - ref).abs() <= step * ref.abs() + 2 * SUM * mag).all())
    n = 1 + T // 8                               # rows of one strand: each adds a rounding
    tol = (n + 64) * 2.0 ** -24
    assert bool(((dg.to(F64) - (D * xh).sum(0)).abs() <= tol * (D * xh).abs().sum(0) + 1e-30).all())
    assert bool(((db.to(F64) - D.sum(0)).abs() <= tol * D.abs().sum(0) + 1e-30).all())


def test_backward_formula_against_differences():
    # the formula that test_backward holds the kernel to, against differences of the
    # definition (fp64 on the CPU: step h, error O(h^2))
    rng = np.random.default_rng(0)
    x, gamma, dy = rng.standard_normal(64), 1 + 0.2 * rng.standard_normal(64), rng.standard_normal(64)

    def f(v):
        return float((gamma * (v - v.mean()) / np.sqrt(v.var() + 1e-5) * dy).sum())
    mu, r = x.mean(), (x.var() + 1e-5) ** -0.5
    xh, a = (x - mu) * r, gamma * dy
    dx = r * (a - a.mean() - xh * (a * xh).mean())
    h = 1e-5
    num = np.array([(f(x + h * e) - f(x - h * e)) / (2 * h) for e in np.eye(64)])
    assert np.abs(num - dx).max() <= 1e-8
    # ... and the kernel on the same numbers: x, gamma and dy representable in its types
    xt = torch.from_numpy(x).to(DEV, F32)[None]
    dyt = torch.from_numpy(dy).to(DEV, BF)[None]
    dy = dyt[0].double().cpu().numpy()
    gt = torch.from_numpy(gamma).to(DEV, F32)
    _, mean, rstd = _forward(xt, gt, None)
    out, _, _ = _backward(dyt, xt, gt, mean, rstd, None)
    num = np.array([(f(x + h * e) - f(x - h * e)) / (2 * h) for e in np.eye(64)])
    assert np.abs(out[0].double().cpu().numpy() - num).max() <= 1e-5


def test_backward_repeats_bit_for_bit_and_adds_in_place():
    x, gamma, _, dy, res = _norm_inputs(1500, 2112, F32, seed=3)
    _, mean, rstd = _forward(x, gamma, None)
    a = _backward(dy, x, gamma, mean, rstd, res)
    b = _backward(dy, x, gamma, mean, rstd, res)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    buf = res.clone()
    c = _backward(dy, x, gamma, mean, rstd, buf, dx=buf)     # dres is dx's own buffer
    assert c[0] is buf and torch.equal(buf, a[0])


def test_a_bad_row_stays_alone():
    x, gamma, beta, dy, _ = _norm_inputs(20, 256, BF)
    y0, _, _ = _forward(x, gamma, beta)
    x[7, 3], x[11, 200] = float("nan"), float("inf")
    y, mean, rstd = _forward(x, gamma, beta)
    keep = [t for t in range(20) if t not in (7, 11)]
    assert torch.equal(y[keep], y0[keep]) and bool(torch.isnan(y[[7, 11]]).all())
    dx, _, _ = _backward(dy, x, gamma, mean, rstd, None)
    assert bool(torch.isfinite(dx[keep]).all())


def test_empty_batch():
    e = torch.empty(0, 128, device=DEV)
    g = torch.ones(128, device=DEV)
    B.moe_layer_norm(e, g, None, 1e-5, e.to(BF))
    dg, db = torch.full((128,), 3.0, device=DEV), torch.full((128,), 3.0, device=DEV)
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    B.moe_layer_norm_backward(e.to(BF), e, g, e[:, 0].contiguous(), e[:, 0].contiguous(), None, e, dg, db, ws)
    assert not bool(dg.any()) and not bool(db.any())
    q, s = B.moe_checkpoint_pack(e.to(BF))
    assert q.shape == (0, 128) and s.shape == (0, 1) and B.moe_checkpoint_unpack(q, s).shape == (0, 128)


def test_other_stream_and_graph():
    x, gamma, beta, dy, _ = _norm_inputs(64, 512, F32)
    y0, m0, r0 = _forward(x, gamma, beta)
    d0 = _backward(dy, x, gamma, m0, r0, None)
    y, mean, rstd = torch.empty_like(y0), torch.empty_like(m0), torch.empty_like(r0)
    dx, dg, db = (torch.empty_like(t) for t in d0)
    ws = torch.zeros(B.moe_layer_norm_backward_workspace_bytes(64, 512), dtype=torch.uint8, device=DEV)

    def both(st=None):
        B.moe_layer_norm(x, gamma, beta, 1e-5, y, mean, rstd, stream=st)
        B.moe_layer_norm_backward(dy, x, gamma, mean, rstd, None, dx, dg, db, ws, stream=st)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    both(s)
    s.synchronize()
    assert torch.equal(y, y0) and torch.equal(dx, d0[0]) and torch.equal(dg, d0[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    x.mul_(0.5)                                  # the graph reads its inputs anew
    g.replay()
    torch.cuda.synchronize()
    y1, m1, r1 = _forward(x, gamma, beta)
    d1 = _backward(dy, x, gamma, m1, r1, None)
    assert torch.equal(y, y1) and torch.equal(dx, d1[0]) and torch.equal(db, d1[2])


# ------------------------------------------------------------------------- 8-bit checkpoint
def _pack_reference(x):
    """Values and exponents of the format, in 64 bits on the CPU."""
    X = x.double().cpu().numpy()
    rows, n = X.shape
    nb = -(-n // 128)
    V = np.zeros((rows, nb, 128))
    V.reshape(rows, nb * 128)[:, :n] = X
    amax = np.nanmax(np.abs(V), axis=2)
    k = np.zeros((rows, nb))
    for i in np.ndindex(amax.shape):
        a = amax[i]
        if np.isinf(a):
            k[i] = 127
        elif a > 0:
            c = int(np.floor(np.log2(a))) - 10
            while a > 448 * 2.0 ** c:
                c += 1
            k[i] = min(max(c, -124), 127)
    with np.errstate(divide="ignore", invalid="ignore"):
        S = V / np.exp2(k)[..., None]
        lead = np.floor(np.log2(np.abs(S)))
        lead = np.where(np.isfinite(lead), lead, 0.0)
        step = np.exp2(np.maximum(lead, -6) - 3)
        Q = np.clip(np.rint(S / step) * step, -448, 448)
        Q = np.where(np.isnan(S), np.nan, Q)
        back = Q * np.exp2(k)[..., None]
        back = np.where(np.abs(back) > 3.39e38, np.sign(Q) * np.inf, back)
    return Q.reshape(rows, nb * 128)[:, :n], back.reshape(rows, nb * 128)[:, :n], k


@pytest.mark.parametrize("rows,n", [(1, 64), (5, 128), (37, 192), (3, 960), (64, 2112), (129, 7168), (2, 16384)])
def test_checkpoint_is_exact(rows, n):
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn(rows, n, generator=g, device=DEV) * torch.exp(6 * torch.randn(rows, 1, generator=g, device=DEV))
    x = x.to(BF)
    x[0, :64] = 0.0
    q, s = B.moe_checkpoint_pack(x)
    out = B.moe_checkpoint_unpack(q, s)
    Q, back, k = _pack_reference(x)
    assert np.array_equal(s.cpu().numpy(), k)
    assert np.array_equal(q.cpu().view(torch.float8_e4m3fn).double().numpy(), Q)
    assert np.array_equal(out.double().cpu().numpy(), back)
    if n % 128 == 0:                              # the layer's own activation format
        assert torch.equal(out, B.moe_quantize_rows_fp8(x))


def test_checkpoint_edges():
    x = torch.zeros(8, 128, dtype=BF, device=DEV)
    x[0, 0], x[0, 1] = 448.0, -1.0                # the maximum on the border: k = 0
    x[1, 0] = 450.0                               # above it (450 is bf16): k = 1
    x[2, 5] = 1e-38                               # the lowest exponents
    x[3, 9] = 2.0 ** -133                         # a bf16 subnormal
    x[4, 0], x[4, 1] = float("inf"), 3.0
    x[5, 0], x[5, 1] = float("nan"), 3.0
    x[6] = torch.finfo(BF).max
    x[7, 3] = -torch.finfo(BF).max
    q, s = B.moe_checkpoint_pack(x)
    out = B.moe_checkpoint_unpack(q, s)
    Q, back, k = _pack_reference(x)
    assert np.array_equal(s.cpu().numpy(), k)
    np.testing.assert_array_equal(out.double().cpu().numpy(), back)
    assert float(out[4, 0]) == float("inf") and bool(torch.isnan(out[5, 0])) and float(out[5, 1]) == 3.0


def test_checkpoint_offsets_past_32_bits():
    # rows past 2^31 elements: 300,000 rows of 7168 are 2.15e9 of them
    rows, n = 300_000, 7168
    x = torch.zeros(rows, n, dtype=BF, device=DEV)
    x[-1] = torch.arange(n, device=DEV).to(BF)
    q, s = B.moe_checkpoint_pack(x)
    out = B.moe_checkpoint_unpack(q, s)
    _, back, k = _pack_reference(x[-1:])
    assert np.array_equal(out[-1:].double().cpu().numpy(), back) and np.array_equal(s[-1:].cpu().numpy(), k)
    assert not bool(out[:-1].any())
