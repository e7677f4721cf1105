"""Orthogonalised updates on the GPU: how far off before the result's rounding, for numbers of steps and
coefficients other than the default ones, and the figures that the header states.

That rounding is averaged away as in test_gpu_orthogonalize_sides.py: `out` is called for with N scales 2^(j / N),
which leaves 2^-8 / sqrt(3 N) (1 + 5 / sqrt(k)) of a matrix of k entries.

Tolerances.  The operands' roundings are restated here, in fp32: X, A and a I + P (P for matrices that one launch
takes) to fp16 at their powers of two, X carried in two numbers (there in fp32).  The kernel's roundings are of
the same sizes but fall differently, as its sums are added in another order; over random matrices the largest error is up to
three times the median one, so three times the largest restated error of 16 matrices is allowed.  Sums: fp32
products here round to nearest; the tensor cores cut off, after aligning to the largest term, with an error of up to
2^-22 to 2^-23 where fp32's is 2^-24, and with a bias: eight times what plain fp32 makes of the formula is allowed on top.
(Directions that a matrix of low rank lacks grow by a in every step: with ten steps plain fp32 is 1e-2 off.)"""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ABC = (3.4445, -4.7750, 2.0315)
SX, SA = 4096.0, 512.0
N = 32


def _matrices(Bn, R, C, kind, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    k = min(R, C)
    if kind == "flat":
        return r(Bn, R, C)
    if kind in ("low", "one"):
        q = max(1, k // 16) if kind == "low" else 1
        return r(Bn, R, q) @ r(Bn, q, C)
    fall = torch.arange(1, k + 1, device=DEV, dtype=F32) ** -1.0
    return (r(Bn, R, k) * fall) @ r(Bn, k, C) + 0.01 * r(Bn, R, C)


def _formula(u, coeffs, dt):
    x = u.to(dt)
    x = x.mT if u.shape[1] > u.shape[2] else x
    x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    for a, b, c in coeffs:
        A = x @ x.mT
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.mT if u.shape[1] > u.shape[2] else x


def _half(t):
    return t.to(torch.float16).to(F32)


def _restated(u, coeffs):
    x = u.mT if u.shape[1] > u.shape[2] else u
    m, n = x.shape[1:]
    one_launch, few = m <= 128 and n <= 8 * 384, m <= 64
    x = x * (SX / torch.linalg.vector_norm(x.to(F64), dim=(1, 2), keepdim=True)).to(F32)
    eye = torch.eye(m, device=DEV)

    def times(s, t):                            # operands in two numbers where there are few
        h, k = _half(s), _half(t)
        return h @ k + h @ _half(t - k) + _half(s - h) @ k
    for i, (a, b, c) in enumerate(coeffs):
        h = _half(x)
        if few and one_launch:
            A = times(x, x.mT) * (SA / SX ** 2)
            x = a * x + times(b * A + c / SA * times(A, A), x) / SA
            continue
        A = (h @ h.mT) * (SA / SX ** 2)
        A, S = (A, times(A, A)) if few else (_half(A), _half(A) @ _half(A))
        P = b * A + c / SA * S
        if one_launch:
            x = a * x + _half(P) @ h / SA
            continue
        low = _half((x - h) * 2048.0) / 2048.0 if i == 0 or i + 1 < len(coeffs) else 0.0
        P = P + a * SA * eye
        x = (_half(P) @ h + (_half(P - _half(P)) @ h if few else 0.0)) / SA + a * low
    x = x / SX
    return x.mT if u.shape[1] > u.shape[2] else x


def _off(x, ref):
    return float((torch.linalg.vector_norm(x.to(F64) - ref, dim=(1, 2)) / torch.linalg.vector_norm(ref, dim=(1, 2))).max())


def _mean(g, coeffs):
    ws = torch.zeros(B.moe_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device=DEV)
    out, mean = torch.empty(g.shape, device=DEV, dtype=BF), torch.zeros(g.shape, device=DEV, dtype=F64)
    for j in range(N):
        s = torch.tensor(2.0 ** (j / N), dtype=F32).item()
        B.moe_orthogonalize(g, out, ws, scale=s, steps=len(coeffs), coeffs=None if all(c == ABC for c in coeffs) else coeffs)
        mean += out.to(F64) / s
    assert B.moe_read_status(ws) == 0
    return mean / N


def _left(g):
    return 2.0 ** -8 / (3 * N) ** 0.5 * (1 + 5 / (g.shape[1] * g.shape[2]) ** 0.5)


# a first step that lifts small singular values, and gentler ones behind it
LIFT = [(8.29, -23.6, 17.3), (4.1, -2.95, 0.53), (3.95, -2.91, 0.53), (3.3, -2.5, 0.48), (2.3, -1.6, 0.42)]
SHAPES = [(16, 48, 48), (16, 5, 700), (16, 16, 3200), (16, 100, 100), (16, 128, 256), (16, 700, 90), (16, 100, 5000), (16, 300, 520),
          (8, 800, 600)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["flat", "fall", "low", "one"])
@pytest.mark.parametrize("coeffs", [[ABC] * 8, [ABC] * 10, LIFT], ids=["8", "10", "lift"])
def test_steps_and_coefficients(shape, kind, coeffs):
    g = _matrices(*shape, kind)
    ref = _formula(g, coeffs, F64)
    tol = 3 * _off(_restated(g, coeffs), ref) + 8 * _off(_formula(g, coeffs, F32), ref) + _left(g)
    assert _off(_mean(g, coeffs), ref) <= tol


# What the header states for the default coefficients and five steps, above 64 on the smaller side.
STATED = 3e-3


@pytest.mark.parametrize("shape", [(32, 65, 65), (32, 65, 300), (32, 100, 100), (32, 128, 256), (16, 90, 3000), (16, 66, 5000), (8, 100, 7168),
                                   (16, 129, 129), (8, 300, 520), (4, 800, 600), (2, 1088, 2112), (1, 2048, 4096)])
@pytest.mark.parametrize("kind", ["flat", "fall", "low", "one"])
def test_the_stated_accuracy(shape, kind):
    g = _matrices(*shape, kind)
    ref = _formula(g, [ABC] * 5, F64)
    assert _off(_mean(g, [ABC] * 5), ref) <= STATED + _left(g)


# The last sizes of one launch (a cluster's CTAs all full but for a column) and the first of the other one; the borders
# between operands in one and in two numbers.
@pytest.mark.parametrize("shape", [(8, 128, 3071), (8, 3071, 128), (8, 120, 3073), (8, 3073, 128), (16, 64, 3071), (16, 3073, 64), (16, 65, 3071),
                                   (16, 64, 384), (16, 385, 64), (16, 65, 385), (16, 128, 768), (16, 769, 128)])
@pytest.mark.parametrize("kind", ["flat", "one"])
def test_at_the_borders_of_the_ways(shape, kind):
    g = _matrices(*shape, kind)
    ref = _formula(g, [ABC] * 5, F64)
    few, longer = min(shape[1:]) <= 64, max(shape[1:]) > 8 * 384
    assert _off(_mean(g, [ABC] * 5), ref) <= (STATED if not few else 1.4e-3 if longer else 3e-4) + _left(g)
