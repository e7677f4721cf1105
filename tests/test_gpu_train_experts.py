"""The expert FFN's backward pass on the GPU against its formulas in 64 bits.

Tolerances.  dg, du and hw are rounded to bf16 once (2^-8 of each value at most) before the
second products, whose sums and the result's own rounding (2^-8) follow: an element of dX or
of a weight gradient is off by at most 2^-8 |result| + 2^-8 (sum of its terms' magnitudes),
and a quarter more of the latter for the fp32 sums of g, u and p.  d topk_w is fp32: a tensor-
core sum of n terms, 16 at a time, cuts each partial sum by 2^-23 of its terms' magnitudes at
most, which reaches <p, h> through p, g and u."""
import numpy as np
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
HALF = 2.0 ** -8


def _problem(T, H, E, K, I, packed, seed=0, idx=None, scale=0.04):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    p = dict(T=T, H=H, E=E, K=K, I=I)
    x = r(T, H).to(BF)
    p["x"], p["xs"] = B.moe_checkpoint_pack(x) if packed else (x, None)
    p["xv"] = B.moe_checkpoint_unpack(p["x"], p["xs"]) if packed else x
    p["dY"] = (0.1 * r(T, H)).to(BF)
    p["W1"], p["W3"] = (scale * r(E, H, I)).to(BF), (scale * r(E, H, I)).to(BF)
    p["W2"] = (scale * r(E, I, H)).to(BF)
    if idx is None:
        idx = torch.rand(T, E, generator=g, device=DEV).topk(K, dim=1).indices
    p["idx"] = idx.to(I32).contiguous()
    p["w"] = (0.1 + torch.rand(T, K, generator=g, device=DEV))
    dispatch(p)
    return p


def dispatch(p):
    T, H, E, K = (p[k] for k in "THEK")
    n = lambda *s: torch.empty(*s, dtype=I32, device=DEV)
    p["counts"], p["offsets"], p["slot"] = n(E), n(E + 1), n(T, K)
    ws = torch.zeros(B.moe_workspace_bytes(T, H, E, K, p["I"], 0), dtype=torch.uint8, device=DEV)
    B.moe_dispatch(p["xv"], p["idx"], E, p["counts"], p["offsets"], n(T * K), p["slot"],
                   torch.empty(T * K, H, dtype=BF, device=DEV), None, ws)


def outputs(p, fill=7.0):
    T, H, E, K, I = (p[k] for k in "THEKI")
    f = lambda *s, t=BF: torch.full(s, fill, dtype=t, device=DEV)
    return dict(dX=f(T, H), dw=f(T, K, t=F32), dW1=f(E, H, I), dW3=f(E, H, I), dW2=f(E, I, H))


def workspace(p):
    n = B.moe_expert_ffn_backward_workspace_bytes(*(p[k] for k in "THEKI"))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)    # NaN wherever nothing is written
    ws[:256] = 0
    return ws


def backward(p, o=None, ws=None, w="given", stream=None):
    o = outputs(p) if o is None else o
    ws = workspace(p) if ws is None else ws
    B.moe_expert_ffn_backward(p["x"], p["xs"], p["dY"], p["offsets"], p["slot"],
                              p["w"] if w == "given" else None, p["W1"], p["W3"], p["W2"], o["dX"], o["dw"],
                              o["dW1"], o["dW3"], o["dW2"], ws, stream=stream)
    return o, ws


def reference(p, ones=False):
    """Gradients and, for each, the sum of its terms' magnitudes (64 bits)."""
    T, H, E, K, I = (p[k] for k in "THEKI")
    x, d = p["xv"].to(F64), p["dY"].to(F64)
    w = torch.ones(T, K, dtype=F64, device=DEV) if ones else p["w"].to(F64)
    z = lambda *s: torch.zeros(*s, dtype=F64, device=DEV)
    ref = dict(dX=z(T, H), dw=z(T, K), dW1=z(E, H, I), dW3=z(E, H, I), dW2=z(E, I, H))
    mag = {k: torch.zeros_like(v) for k, v in ref.items()}
    cut = (H / 16 + 32) * 2.0 ** -23
    for e in range(E):
        t, j = (p["idx"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        W1, W3, W2 = (p[n][e].to(F64) for n in ("W1", "W3", "W2"))
        xe, de, we = x[t], d[t], w[t, j][:, None]
        g, u, q = xe @ W1, xe @ W3, de @ W2.T
        s = torch.sigmoid(g)
        h = g * s * u
        dg, du = we * q * u * s * (1 + g * (1 - s)), we * q * g * s
        ref["dw"][t, j] = (q * h).sum(1)
        ref["dX"].index_add_(0, t, dg @ W1.T + du @ W3.T)
        ref["dW1"][e], ref["dW3"][e], ref["dW2"][e] = xe.T @ dg, xe.T @ du, (we * h).T @ de
        mag["dX"].index_add_(0, t, dg.abs() @ W1.T.abs() + du.abs() @ W3.T.abs())
        mag["dW1"][e], mag["dW3"][e] = xe.T.abs() @ dg.abs(), xe.T.abs() @ du.abs()
        mag["dW2"][e] = (we * h).T.abs() @ de.abs()
        ga, ua, qa = xe.abs() @ W1.abs(), xe.abs() @ W3.abs(), de.abs() @ W2.T.abs()
        mag["dw"][t, j] = cut * (qa * h.abs() + q.abs() * (1.1 * ga * u.abs() + (g * s).abs() * ua)).sum(1)
    return ref, mag


def check(o, ref, mag):
    for k in ("dX", "dW1", "dW3", "dW2"):
        got = o[k].to(F64)
        tol = HALF * ref[k].abs() + 1.25 * HALF * mag[k]
        assert bool(((got - ref[k]).abs() <= tol).all()), k
        n = float(ref[k].norm())
        assert float((got - ref[k]).norm()) <= HALF * n, k
    assert bool(((o["dw"].to(F64) - ref["dw"]).abs() <= mag["dw"] + 1e-30).all())


SHAPES = [(1, 64, 1, 1, 64), (1, 128, 9, 4, 320), (16, 256, 16, 2, 128), (45, 320, 5, 3, 192), (300, 512, 7, 2, 448),
          (777, 576, 24, 3, 1088), (64, 7168, 4, 2, 256), (1200, 192, 2, 2, 2112), (130, 1088, 70, 8, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("packed", [False, True])
def test_gradients(shape, packed):
    p = _problem(*shape, packed)
    o, ws = backward(p)
    assert B.moe_read_status(ws) == 0
    check(o, *reference(p))


def test_formulas_against_differences():
    # the formulas of reference() against differences of sum(Y dY), one expert, 64 bits
    rng = np.random.default_rng(1)
    x, d = rng.standard_normal(5), rng.standard_normal(5)
    W1, W3, W2 = rng.standard_normal((5, 4)), rng.standard_normal((5, 4)), rng.standard_normal((4, 5))
    w = 0.7

    def f(x, W1, W3, W2, w):
        g, u = x @ W1, x @ W3
        return w * float(((g / (1 + np.exp(-g)) * u) @ W2) @ d)
    g, u, q = x @ W1, x @ W3, W2 @ d
    s = 1 / (1 + np.exp(-g))
    h = g * s * u
    dg, du = w * q * u * s * (1 + g * (1 - s)), w * q * g * s
    want = [W1 @ dg + W3 @ du, np.outer(x, dg), np.outer(x, du), np.outer(w * h, d), np.array(q @ h)]
    args = [x, W1, W3, W2, np.array(w)]
    for k in range(5):
        num = np.zeros_like(args[k])
        for i in np.ndindex(args[k].shape):
            a = [v.copy() for v in args]
            b = [v.copy() for v in args]
            a[k][i] += 1e-6
            b[k][i] -= 1e-6
            num[i] = (f(*a) - f(*b)) / 2e-6
        assert np.abs(num - want[k]).max() <= 1e-7 * max(1.0, np.abs(want[k]).max())


def test_one_expert_takes_all_and_others_none():
    T, E = 600, 6
    idx = torch.full((T, 1), 2, device=DEV)
    p = _problem(T, 256, E, 1, 192, True, idx=idx)
    o, _ = backward(p)
    check(o, *reference(p))
    for e in (0, 1, 3, 4, 5):
        assert not bool(o["dW1"][e].any()) and not bool(o["dW3"][e].any()) and not bool(o["dW2"][e].any())


def test_group_sizes_around_the_tiles():
    # rows per expert on and beside the 64-row padding and the 256-row tiles
    sizes = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 320, 0, 511, 513, 0]
    idx = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(sizes))
    idx = idx[torch.randperm(idx.numel(), generator=torch.Generator().manual_seed(0))].to(DEV)[:, None]
    p = _problem(idx.numel(), 192, len(sizes), 1, 320, False, idx=idx)
    assert p["counts"].tolist() == sizes
    o, _ = backward(p)
    check(o, *reference(p))


def test_without_weights_and_without_their_gradient():
    # the shared expert: one group, every token once, weight 1
    T = 77
    p = _problem(T, 256, 1, 1, 128, True, idx=torch.zeros(T, 1, device=DEV))
    assert p["slot"].flatten().tolist() == list(range(T))
    o, _ = backward(p, w="none")
    check(o, *reference(p, ones=True))
    q = outputs(p)
    q2 = dict(q, dw=None)
    backward(p, o=q2, w="none")
    assert all(torch.equal(q[k], o[k]) for k in ("dX", "dW1", "dW3", "dW2"))


def test_rejected_pairs_have_no_gradient():
    p = _problem(90, 256, 8, 3, 128, False, seed=5)
    p["idx"][4, 1], p["idx"][50, 0], p["idx"][89] = -1, 8, 100
    dispatch(p)
    o, _ = backward(p)
    ref, mag = reference(p)
    check(o, ref, mag)
    assert float(o["dw"][4, 1]) == 0 and float(o["dw"][50, 0]) == 0 and not bool(o["dw"][89].any())
    assert not bool(o["dX"][89].any())


@pytest.mark.parametrize("bad", ["decreasing", "past_rows", "negative"])
def test_bad_offsets_are_refused_on_the_device(bad):
    p = _problem(40, 256, 8, 2, 128, False)
    good = p["offsets"].clone()
    off = good.cpu().numpy()
    if bad == "decreasing":
        off[3], off[4] = off[4] + 1, off[3]
    elif bad == "past_rows":
        off[-1] = 81
    else:
        off[0] = -16
    p["offsets"] = torch.from_numpy(off).to(DEV)
    o, ws = backward(p)
    assert B.moe_read_status(ws) == -1
    assert all(bool((v == 7).all()) for v in o.values())
    p["offsets"] = good
    o, ws = backward(p, ws=ws)
    assert B.moe_read_status(ws) == 0
    check(o, *reference(p))


def test_repeats_bit_for_bit_on_other_streams_and_in_a_graph():
    p = _problem(300, 512, 7, 2, 448, True)
    a, ws = backward(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b, _ = backward(p, stream=s)
    s.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
    g = torch.cuda.CUDAGraph()
    c = outputs(p)
    with torch.cuda.graph(g):
        backward(p, o=c, ws=ws)
    p["dY"].neg_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], -c[k]) for k in a)


def test_a_wait_that_runs_out_is_reported():
    p = _problem(45, 256, 8, 2, 128, False)
    B.moe_debug_set_wait_limit(50_000_000, inject_stall=1)       # 50 ms
    try:
        _, ws = backward(p)
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    o, ws = backward(p, ws=ws)
    assert B.moe_read_status(ws) == 0
    check(o, *reference(p))


def test_empty_batch():
    e = lambda *s, t=BF: torch.empty(*s, dtype=t, device=DEV)
    W = torch.ones(2, 64, 64, dtype=BF, device=DEV)
    d = [torch.ones_like(W) for _ in range(3)]
    ws = torch.zeros(B.moe_expert_ffn_backward_workspace_bytes(0, 64, 2, 1, 64), dtype=torch.uint8, device=DEV)
    B.moe_expert_ffn_backward(e(0, 64), None, e(0, 64), torch.zeros(3, dtype=I32, device=DEV), e(0, 1, t=I32), None,
                              W, W, W, e(0, 64), None, d[0], d[1], d[2], ws)
    assert not any(bool(v.any()) for v in d)


@pytest.mark.parametrize("shape", [(16, 64, 256, 4, 64), (16, 64, 257, 4, 64), (1016, 64, 8, 1, 64), (1017, 64, 8, 1, 64)])
def test_both_sides_of_the_rule_on_where_the_plan_is_made(shape):
    p = _problem(*shape, False)
    o, ws = backward(p)
    assert B.moe_read_status(ws) == 0
    check(o, *reference(p))
    off = p["offsets"].cpu().numpy()
    off[-1] = shape[0] * shape[3] + 1
    good, p["offsets"] = p["offsets"], torch.from_numpy(off).to(DEV)
    o, _ = backward(p, ws=ws)
    assert B.moe_read_status(ws) == -1
    assert all(bool((v == 7).all()) for v in o.values())
    p["offsets"] = good
    o, _ = backward(p, ws=ws)
    assert B.moe_read_status(ws) == 0
    check(o, *reference(p))
