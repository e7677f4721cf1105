"""Routing from given logits and its gradient on the GPU against the definition in 64 bits.
The selection has to be equal; weights and gradients are fp32 (or rounded once to bf16)."""
import numpy as np
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
MASKED = float(torch.finfo(BF).min)
# fp32 scores: exp, sum and division are off by a few steps of 2^-24 each (32 terms a lane
# and 5 levels in a softmax's sum)
W_REL = 64 * 2.0 ** -24


def _scores(l, scoring):
    off = l <= MASKED
    if scoring == "sigmoid":
        s = 1 / (1 + np.exp(-l))
    else:
        m = np.max(np.where(off, -1e300, l), axis=1, keepdims=True)
        z = np.where(off, 0.0, np.exp(np.where(off, 0.0, l) - np.where(m > -1e299, m, 0.0)))
        tot = z.sum(1, keepdims=True)
        s = z / np.where(tot > 0, tot, 1.0)
    return np.where(off, 0.0, s)


def _reference(l, bias, K, scoring="sigmoid", n_group=1, topk_group=1, group_top=1, renorm=True):
    l = l.astype(np.float64)
    T, E = l.shape
    with np.errstate(over="ignore"):
        s = _scores(l, scoring)
    sel = s + (0.0 if bias is None else bias.astype(np.float64))
    if bias is None and group_top == 1:
        sel = l.copy()                              # the same order, exactly
    sel = np.where(l <= MASKED, -1e300, sel)
    G = E // n_group
    if n_group > 1:
        best = -np.sort(-sel.reshape(T, n_group, G), axis=2)[:, :, :group_top].sum(2)
        drop = np.argsort(-best, axis=1, kind="stable")[:, topk_group:]
        gone = np.zeros((T, n_group), bool)
        gone[np.arange(T)[:, None], drop] = True
        sel = np.where(np.repeat(gone, G, axis=1), -np.inf, sel)
    idx = np.argsort(-sel, axis=1, kind="stable")[:, :K]
    w = s[np.arange(T)[:, None], idx]
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
    return idx, w


def _route(logits, bias, K, **opts):
    T = logits.shape[0]
    idx = torch.full((T, K), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, K), -7.0, device=DEV)
    B.moe_route_logits(logits, bias, K, opts or None, idx, w)
    return idx, w


def _check(logits, bias, K, **opts):
    idx, w = _route(logits, bias, K, **opts)
    b = None if bias is None else bias.cpu().numpy()
    ri, rw = _reference(logits.double().cpu().numpy(), b, K, **opts)
    got = idx.cpu().numpy()
    bad = np.nonzero((got != ri).any(1))[0]
    assert bad.size == 0, (bad[:5], got[bad[:3]], ri[bad[:3]])
    assert bool(np.all(np.abs(w.double().cpu().numpy() - rw) <= W_REL * rw + 1e-37))
    return idx, w


def _logits(T, E, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (1.7 * torch.randn(T, E, generator=g, device=DEV)).to(dtype)


CASES = [
    (60, 200, 8, dict(n_group=8, topk_group=3, group_top=2)),
    (40, 1020, 9, dict(n_group=17, topk_group=4, group_top=2)),
    (40, 72, 4, dict(n_group=12, topk_group=2, group_top=2)),
    (1, 1, 1, dict()),
    (3, 8, 8, dict(scoring="softmax")),
    (45, 16, 2, dict()),
    (7, 33, 5, dict(scoring="softmax", renorm=False)),
    (2, 256, 8, dict(n_group=8, topk_group=4, group_top=2)),
    (515, 256, 8, dict(n_group=8, topk_group=4, group_top=2)),
    (300, 160, 6, dict(scoring="softmax", n_group=8, topk_group=3, group_top=1, renorm=False)),
    (200, 96, 4, dict(scoring="softmax", n_group=32, topk_group=5, group_top=2)),
    (64, 512, 32, dict(renorm=False)),
    (40, 1000, 31, dict(scoring="softmax")),
    (33, 1024, 32, dict(n_group=2, topk_group=1, group_top=2)),
    (90, 274, 15, dict(scoring="softmax", n_group=2, topk_group=1, group_top=2, renorm=False)),
    (70, 512, 16, dict(n_group=8, topk_group=1, group_top=2)),
    (50, 960, 20, dict(scoring="softmax", n_group=32, topk_group=2, group_top=1)),
]


@pytest.mark.parametrize("T,E,K,opts", CASES)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("with_bias", [False, True])
def test_forward(T, E, K, opts, dtype, with_bias):
    bias = None
    if with_bias:
        bias = 0.2 * torch.rand(E, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) - 0.1
    _check(_logits(T, E, dtype), bias, K, **opts)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("opts", [dict(), dict(n_group=8, topk_group=3, group_top=2)])
def test_ties_and_near_ties(scoring, opts):
    # few distinct logits and biases: equal sums go to the lower index; and logits a few
    # steps apart whose scores an fp32 sum with the bias cannot tell apart
    rng = np.random.default_rng(4)
    T, E, K = 400, 64, 8
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)
    b = rng.choice([0.0, 0.05], E).astype(np.float32)
    _check(torch.from_numpy(l).to(DEV), torch.from_numpy(b).to(DEV), K, scoring=scoring, **opts)
    _check(torch.from_numpy(l).to(DEV), None, K, scoring=scoring, **opts)
    near = (1.0 + 2.0 ** -22 * rng.integers(0, 40, (T, E))).astype(np.float32)
    const = torch.full((E,), 0.07, device=DEV)
    _check(torch.from_numpy(near).to(DEV), const, K, scoring=scoring, **opts)
    _check(torch.from_numpy(near).to(DEV), None, K, scoring=scoring, **opts)
    # opposite zeros are equal
    z = torch.zeros(2, E, device=DEV)
    z[:, ::2] = -0.0
    idx, _ = _check(z, None, K, scoring=scoring, **opts)
    assert idx[0].tolist() == list(range(K))


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("low", ["inf", "bf16", "fp32"])
@pytest.mark.parametrize("opts", [dict(), dict(n_group=4, topk_group=2, group_top=2),
                                  dict(n_group=4, topk_group=2, group_top=1)])
def test_masks(scoring, with_bias, low, opts):
    T, E, K = 64, 32, 6
    l = _logits(T, E, F32, seed=2)
    m = {"inf": -float("inf"), "bf16": MASKED, "fp32": float(torch.finfo(F32).min)}[low]
    g = torch.Generator(device=DEV).manual_seed(5)
    l[torch.rand(T, E, generator=g, device=DEV) < 0.6] = m
    l[3] = m                                        # nothing left
    l[4] = m
    l[4, 17] = -3.0                                 # one left
    l[5] = -1e35                                    # far down, not masked
    l[5, 3] = m
    bias = -0.5 * torch.rand(E, generator=g, device=DEV) if with_bias else None
    idx, w = _check(l, bias, K, scoring=scoring, **opts)
    assert not bool(w[3].any()) and bool(torch.isfinite(w).all())
    assert sorted(set(idx[3].tolist())) == sorted(idx[3].tolist())
    assert float(w[4].sum()) == 1.0 and int(idx[4, 0]) == 17


def test_bias_of_minus_infinity_and_large_bias():
    l = _logits(50, 64, F32, seed=3)
    b = torch.zeros(64, device=DEV)
    b[::3] = -float("inf")
    b[1] = 1e4
    idx, _ = _check(l, b, 8)
    assert bool((idx[:, 0] == 1).all())
    half = torch.zeros(40, device=DEV)
    half[::2] = -float("inf")
    _check(_logits(50, 40, F32, seed=3), half, 32)  # -inf biases have to be taken, by index
    _check(l, b, 8, n_group=8, topk_group=2, group_top=2)


def test_nan_rows_get_distinct_experts():
    l = _logits(8, 40, F32, seed=6)
    l[1, 5] = float("nan")
    l[2] = float("nan")
    l[3, 4] = float("inf")
    for opts in (dict(), dict(scoring="softmax"), dict(n_group=4, topk_group=2, group_top=2)):
        for bias in (None, torch.zeros(40, device=DEV)):
            idx, _ = _route(l, bias, 6, **opts)
            for row in idx.tolist():
                assert len(set(row)) == 6 and min(row) >= 0 and max(row) < 40
            clean = [0, 4, 5, 6, 7]
            ri, _ = _reference(l[clean].double().cpu().numpy(), None, 6, **opts)
            assert np.array_equal(idx[clean].cpu().numpy(), ri)


def _gradient(l, idx, dw, scoring, renorm):
    l = l.double().cpu()
    off = l <= MASKED
    x = l.masked_fill(off, -1e4).requires_grad_(True)
    s = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, 1)
    v = s.masked_fill(off, 0.0).gather(1, idx.long().cpu())
    if renorm:
        t = v.sum(1, keepdim=True)
        v = torch.where(t > 0, v / torch.where(t > 0, t, torch.ones_like(t)), torch.zeros_like(v))
    v.backward(dw.double().cpu())
    return x.grad.masked_fill(off, 0.0)


@pytest.mark.parametrize("T,E,K,opts", CASES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_backward(T, E, K, opts, dtype):
    l = _logits(T, E, dtype, seed=1)
    if E >= 16:
        l[0, 3] = MASKED
    idx, _ = _route(l, None, K, **opts)
    g = torch.Generator(device=DEV).manual_seed(8)
    dw = torch.randn(T, K, generator=g, device=DEV)
    out = torch.full_like(l, 7.0)
    B.moe_route_logits_backward(l, opts or None, idx, dw, out)
    ref = _gradient(l, idx, dw, opts.get("scoring", "sigmoid"), opts.get("renorm", True))
    # terms of size |dw| <= max that may cancel; fp32 throughout, one rounding to the type
    step = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = step * ref.abs() + 2 * W_REL * float(dw.abs().max())
    assert bool(((out.double().cpu() - ref).abs() <= tol).all())


def test_backward_against_differences():
    # the gradient of sum(w dw) with the selection fixed, by differences in 64 bits
    rng = np.random.default_rng(2)
    E, K = 12, 4
    for scoring in ("sigmoid", "softmax"):
        for renorm in (True, False):
            l = rng.standard_normal((1, E)).astype(np.float32)
            idx, _ = _reference(l, None, K, scoring)
            dw = rng.standard_normal((1, K)).astype(np.float32)

            def f(v):
                s = _scores(v, scoring)[0, idx[0]]
                return float(((s / s.sum() if renorm else s) * dw[0]).sum())
            h = 1e-5
            num = np.array([(f(l + h * e) - f(l - h * e)) / (2 * h) for e in np.eye(E)[:, None, :]])
            t = torch.from_numpy(l).to(DEV)
            out = torch.empty_like(t)
            B.moe_route_logits_backward(t, dict(scoring=scoring, renorm=renorm),
                                        torch.from_numpy(idx.astype(np.int32)).to(DEV),
                                        torch.from_numpy(dw).to(DEV), out)
            assert np.abs(out[0].double().cpu().numpy() - num).max() <= 1e-6


def test_backward_rejected_pairs_and_masked_rows():
    l = _logits(6, 24, F32, seed=7)
    l[2] = -float("inf")
    idx, _ = _route(l, None, 4)
    idx[1, 2], idx[4, 0], idx[5] = -1, 24, -3
    dw = torch.ones(6, 4, device=DEV)
    for scoring in ("sigmoid", "softmax"):
        for renorm in (True, False):
            out = torch.full_like(l, 7.0)
            B.moe_route_logits_backward(l, dict(scoring=scoring, renorm=renorm), idx, dw, out)
            assert bool(torch.isfinite(out).all())
            assert not bool(out[2].any()) and not bool(out[5].any())


def test_other_stream_and_graph():
    l = _logits(100, 64, F32)
    bias = torch.linspace(-0.1, 0.1, 64, device=DEV)
    opts = B.MoeRouting.make(n_group=8, topk_group=4, group_top=2)
    i0, w0 = _route(l, bias, 6, n_group=8, topk_group=4, group_top=2)
    idx, w, out = torch.empty_like(i0), torch.empty_like(w0), torch.empty_like(l)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    B.moe_route_logits(l, bias, 6, opts, idx, w, stream=s)
    s.synchronize()
    assert torch.equal(idx, i0) and torch.equal(w, w0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_route_logits(l, bias, 6, opts, idx, w)
        B.moe_route_logits_backward(l, opts, idx, w, out)
    l.neg_()
    g.replay()
    torch.cuda.synchronize()
    i1, w1 = _route(l, bias, 6, n_group=8, topk_group=4, group_top=2)
    ref = torch.empty_like(l)
    B.moe_route_logits_backward(l, opts, i1, w1, ref)
    assert torch.equal(idx, i1) and torch.equal(w, w1) and torch.equal(out, ref)
