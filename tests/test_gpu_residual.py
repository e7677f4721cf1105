"""The branch joined to the residual stream, with its norms and gates, forward and backward, on the
GPU against the definition in 64 bits.

Tolerances.  A bf16 result is off by half a step, 2^-8 of its value, an fp32 one by 2^-24, on top of
what the fp32 sums before it lose: a sum over a row runs in strands of at most 16 terms with a
tree above them, 32 * 2^-24 of the sum of the terms' magnitudes at most (SUM).  Errors are carried
through the formulas as bounds (the names ending in _e)."""
import subprocess
import sys

import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
SUM = 32 * U
EPS = 1e-5


def _inputs(T, H, xt, yt, post, pre, gate, token, beta=True, seed=0, offset=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = (r(T, H) * (0.3 + 2 * torch.rand(T, 1, generator=g, device=DEV)) + offset).to(xt)
    y = (r(T, H) * (0.2 + torch.rand(T, 1, generator=g, device=DEV)) + offset).to(yt)
    p = dict(post=post, pre=pre, alpha=0.75, eps_post=EPS, eps_pre=EPS)
    for end in ("post", "pre"):
        if p[end] != "none":
            p["gamma_" + end] = 1 + 0.2 * r(H)
            if beta:
                p["beta_" + end] = 0.3 * r(H)
    if gate:
        p["gate"] = 0.7 + 0.3 * r(H)
    if token:
        p["gate_token"] = torch.rand(T, generator=g, device=DEV)
        p["gate_token"][0] = 0.0
    dn, dr = (0.1 * r(T, H)).to(BF), (0.2 * r(T, H)).to(xt)
    return x, y, p, dn, dr


def _forward(x, y, p, r=None):
    T, H = x.shape
    r = torch.empty_like(x) if r is None else r
    n = torch.empty(T, H, dtype=BF, device=DEV) if p["pre"] != "none" else None
    stats = torch.full((T, 4), 7.0, device=DEV)
    B.moe_residual_norm(x, y, p, r, n, stats)
    return r, n, stats


def _stat(v, kind):
    if kind == "none":
        return torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
    mu = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return mu, ((v - mu).square().mean(1, keepdim=True) + EPS) ** -0.5


def _normed(v, p, end):
    """-> norm of v and a bound on its error"""
    if p[end] == "none":
        return v, torch.zeros_like(v)
    mu, rs = _stat(v, p[end])
    ga = p["gamma_" + end].to(F64)
    be = p["beta_" + end].to(F64) if p.get("beta_" + end) is not None else torch.zeros_like(ga)
    size = v.abs().amax(1, keepdim=True)
    out = ga * (v - mu) * rs + be
    return out, 4 * SUM * (1 + size * rs) * (ga.abs() * size * rs + be.abs())


def _gates(p, T, H):
    gh = p["gate"].to(F64) if p.get("gate") is not None else torch.ones(H, dtype=F64, device=DEV)
    gt = p["gate_token"].to(F64)[:, None] if p.get("gate_token") is not None else torch.ones(T, 1, dtype=F64, device=DEV)
    return gh, gt


SHAPES = [(1, 64), (3, 256), (45, 320), (19, 512), (9, 576), (33, 1024), (700, 2112), (200, 7168), (3, 8256), (5, 11264),
          (2, 16384)]
KINDS = [("none", "rms", False, False, True), ("rms", "layer", True, False, False), ("layer", "none", False, True, True),
         ("layer", "rms", True, True, True), ("none", "none", True, True, True), ("none", "none", False, False, True),
         ("rms", "none", False, True, True), ("layer", "layer", False, False, False)]
TYPES = [(F32, F32), (BF, F32), (BF, BF), (F32, BF)]


def _check_forward(x, y, p, r, n, stats):
    T, H = x.shape
    Y, X = y.to(F64), x.to(F64)
    b, b_e = _normed(Y, p, "post")
    gh, gt = _gates(p, T, H)
    ref = p["alpha"] * X + gt * gh * b
    tol = (gt * gh).abs() * b_e + 4 * U * (X.abs() + (gt * gh * b).abs())
    assert bool(((r.to(F64) - ref).abs() <= HALF[r.dtype] * (ref.abs() + tol) + tol).all())
    R = r.to(F64)                              # the next norm is that of the stored stream
    for k, (v, end) in enumerate(((Y, "post"), (R, "pre"))):
        mu, rs = _stat(v, p[end])
        size = v.abs().amax(1)
        assert bool(((stats[:, 2 * k].to(F64) - mu[:, 0]).abs() <= SUM * size).all())
        assert bool(((stats[:, 2 * k + 1].to(F64) / rs[:, 0] - 1).abs() <= 2 * SUM * (1 + size * rs[:, 0])).all())
    if n is not None:
        ref, tol = _normed(R, p, "pre")
        assert bool(((n.to(F64) - ref).abs() <= HALF[BF] * ref.abs() + tol).all())


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("xt,yt", TYPES)
def test_forward(T, H, kinds, xt, yt):
    x, y, p, _, _ = _inputs(T, H, xt, yt, *kinds)
    r, n, stats = _forward(x, y, p)
    _check_forward(x, y, p, r, n, stats)
    again = x.clone()                          # in place
    r2, n2, _ = _forward(again, y, p, r=again)
    assert torch.equal(r2, r) and (n is None or torch.equal(n2, n))


def _rounded_stats(y, r, p):
    return torch.cat([torch.cat(_stat(v.to(F64), p[end]), 1) for v, end in ((y, "post"), (r, "pre"))], 1).to(F32)


def _backward(dn, dr, y, r, stats, p, dx=None, wanted=None):
    T, H = r.shape
    dx = torch.empty_like(r) if dx is None else dx
    dy = torch.full((T, H), 7.0, device=DEV).to(BF)
    grads = {k: torch.full_like(v, 7.0) for k, v in p.items() if torch.is_tensor(v) and (wanted is None or k in wanted)}
    ws = torch.zeros(B.moe_residual_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    B.moe_residual_norm_backward(dn if p["pre"] != "none" else None, dr, y, r, stats, p, dx, dy, grads, ws)
    return dx, dy, grads


def _through(a, a_e, h, rs, kind):
    """rstd (a - [layer] mean(a) - h mean(a h)) and a bound on its error"""
    if kind == "none":
        return a, a_e
    m1, m1_e = (a * h).mean(1, keepdim=True), (a_e * h.abs() + (SUM + 8 * U) * (a * h).abs()).mean(1, keepdim=True)
    m0, m0_e = a.mean(1, keepdim=True), (a_e + SUM * a.abs()).mean(1, keepdim=True)
    if kind == "rms":
        m0, m0_e = torch.zeros_like(m0), torch.zeros_like(m0)
    return (rs * (a - m0 - h * m1),
            rs * (a_e + m0_e + h.abs() * m1_e + 8 * U * (a.abs() + m0.abs() + (h * m1).abs())))


def _reference(dn, dr, y, r, stats, p):
    """Gradients for given statistics, each with a bound on an fp32 evaluation's error"""
    T, H = r.shape
    st = stats.to(F64)
    gh, gt = _gates(p, T, H)
    # sums over the rows: a CTA's rows one after the other (at most 8 in these tests), 304 CTAs in 8 strands
    ROWS = (8 + 38 + 16) * U
    o = {}
    d = torch.zeros(T, H, dtype=F64, device=DEV) if dr is None else dr.to(F64)
    d_e = torch.zeros_like(d)
    if p["pre"] != "none":
        e, h, rs = dn.to(F64), (r.to(F64) - st[:, 2:3]) * st[:, 3:4], st[:, 3:4]
        o["gamma_pre"] = ((e * h).sum(0), (ROWS + 4 * U) * (e * h).abs().sum(0))
        o["beta_pre"] = (e.sum(0), ROWS * e.abs().sum(0))
        a = e * p["gamma_pre"].to(F64)
        t, t_e = _through(a, U * a.abs(), h, rs, p["pre"])
        d_e = t_e + 2 * U * (t.abs() + d.abs())
        d = d + t
    v, rs = y.to(F64), torch.ones(T, 1, dtype=F64, device=DEV)
    if p["post"] != "none":
        v, rs = (v - st[:, 0:1]) * st[:, 1:2], st[:, 1:2]
    ga = p["gamma_post"].to(F64) if p.get("gamma_post") is not None else torch.ones(H, dtype=F64, device=DEV)
    be = p["beta_post"].to(F64) if p.get("beta_post") is not None else torch.zeros(H, dtype=F64, device=DEV)
    b = ga * v + be
    s1, s1_e = (gt * d * v).sum(0), (gt.abs() * v.abs() * (d_e + (ROWS + 4 * U) * d.abs())).sum(0)
    s0, s0_e = (gt * d).sum(0), (gt.abs() * (d_e + (ROWS + 2 * U) * d.abs())).sum(0)
    o["gamma_post"] = (gh * s1, gh.abs() * (s1_e + U * s1.abs()))
    o["beta_post"] = (gh * s0, gh.abs() * (s0_e + U * s0.abs()))
    o["gate"] = (ga * s1 + be * s0, ga.abs() * s1_e + be.abs() * s0_e + 3 * U * ((ga * s1).abs() + (be * s0).abs()))
    k = d * gh
    o["gate_token"] = ((k * b).sum(1), (gh.abs() * d_e * (ga * v).abs() + gh.abs() * d_e * be.abs()
                                        + (SUM + 8 * U) * k.abs() * ((ga * v).abs() + be.abs())).sum(1))
    f = k * ga
    dy, dy_e = _through(f, (gh * ga).abs() * d_e + 4 * U * f.abs(), v, rs, p["post"])
    o = {q: w for q, w in o.items() if p.get(q) is not None}
    return (p["alpha"] * d, p["alpha"] * d_e + 2 * U * d.abs()), (gt * dy, gt * dy_e + 2 * U * (gt * dy).abs()), o


def _near(got, ref, tol):
    return bool(((got.to(F64) - ref).abs() <= HALF[got.dtype] * (ref.abs() + tol) + tol).all())


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("with_dr", [True, False])
def test_backward(T, H, kinds, xt, yt, with_dr):
    if not with_dr and kinds[1] == "none":
        pytest.skip("no gradient reaches the stream")
    x, y, p, dn, dr = _inputs(T, H, xt, yt, *kinds)
    dr = dr if with_dr else None
    r, _, _ = _forward(x, y, p)
    stats = _rounded_stats(y, r, p)
    dx, dy, grads = _backward(dn, dr, y, r, stats, p)
    rdx, rdy, ref = _reference(dn, dr, y, r, stats, p)
    assert _near(dx, *rdx) and _near(dy, *rdy)
    assert set(grads) == set(ref)
    for q, g in grads.items():
        assert _near(g, *ref[q]), q
    if with_dr:                                 # over dr, and with no parameter's gradient wanted
        over = dr.clone()
        dx2, dy2, _ = _backward(dn, over, y, r, stats, p, dx=over, wanted=())
        assert torch.equal(dx2, dx) and torch.equal(dy2, dy)


# (up to eight CTAs are a cluster that adds its own column sums; one more and a second launch does)
@pytest.mark.parametrize("T,H", [(T, H) for H in (64, 320) for T in (1, 8, 9, 31, 40, 63, 64, 65)] +
                         [(T, H) for H in (576, 7168, 16384) for T in (1, 2, 3, 6, 8, 9)])
def test_column_gradients_of_few_rows(T, H):
    for kinds in (KINDS[3], KINDS[1], KINDS[4]):
        x, y, p, dn, dr = _inputs(T, H, F32, F32, *kinds)
        r, _, _ = _forward(x, y, p)
        stats = _rounded_stats(y, r, p)
        ref = _reference(dn, dr, y, r, stats, p)[2]
        grads = {k: torch.full_like(v, 7.0) for k, v in p.items() if torch.is_tensor(v)}
        n = B.moe_residual_norm_backward_workspace_bytes(T, H)
        ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=DEV)
        dx, dy = torch.empty_like(r), torch.empty(T, H, device=DEV, dtype=BF)

        def call():
            B.moe_residual_norm_backward(dn if p["pre"] != "none" else None, dr, y, r, stats, p, dx, dy, grads, ws[:n])
        call()
        for q, g in grads.items():
            assert _near(g, *ref[q]), q
        assert bool((ws[n:] == 255).all())
        kept = {q: g.clone() for q, g in grads.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for g in grads.values():
            g.zero_()
        graph.replay()
        assert all(torch.equal(grads[q], kept[q]) for q in kept)


def test_formula_against_differences():
    # the reference's own gradients: central differences of the definition in 64 bits
    T, H = 4, 64
    for kinds in KINDS:
        x, y, p, dn, dr = _inputs(T, H, F32, F32, *kinds)
        x64, y64 = x.to(F64), y.to(F64)
        p64 = {k: v.to(F64) if torch.is_tensor(v) else v for k, v in p.items()}
        dn64, dr64 = dn.to(F64), dr.to(F64)

        def value(x, y, q):
            b, _ = _normed(y, q, "post")
            gh, gt = _gates(q, T, H)
            r = q["alpha"] * x + gt * gh * b
            n, _ = _normed(r, q, "pre")
            return (dr64 * r).sum() + ((dn64 * n).sum() if q["pre"] != "none" else 0.0), r
        _, r = value(x64, y64, p64)
        stats = torch.cat([torch.cat(_stat(v, p[end]), 1) for v, end in ((y64, "post"), (r, "pre"))], 1)
        dx, dy, grads = _reference(dn64, dr64, y64, r, stats, p64)
        g = torch.Generator(device=DEV).manual_seed(5)
        step = 1e-5
        for name, grad in dict(x=dx, y=dy, **grads).items():
            base = x64 if name == "x" else y64 if name == "y" else p64[name]
            v = torch.randn(base.shape, generator=g, device=DEV, dtype=F64)

            def at(s):
                if name == "x":
                    return value(x64 + s * v, y64, p64)[0]
                if name == "y":
                    return value(x64, y64 + s * v, p64)[0]
                return value(x64, y64, {**p64, name: p64[name] + s * v})[0]
            slope = float(at(step) - at(-step)) / (2 * step)
            assert abs(slope - float((grad[0] * v).sum())) <= 1e-6 * (1 + float((grad[0] * v).abs().sum())), (kinds, name)


def test_rows_far_from_zero_and_constant_rows():
    x, y, p, _, _ = _inputs(8, 7168, F32, F32, "layer", "layer", True, False, offset=1000.0)
    y[3] = 5.0                                  # no spread: b = beta
    y[4] = 0.0
    r, n, stats = _forward(x, y, p)
    Y = y.to(F64)
    rs = ((Y - Y.mean(1, keepdim=True)).square().mean(1) + EPS) ** -0.5
    live = [0, 1, 2, 5, 6, 7]
    # the mean is off by SUM * 1000 at most, which moves a spread of >= 0.2 by its square
    assert bool(((stats[:, 1].to(F64) / rs - 1).abs()[live] <= 1e-5).all())
    want = (p["alpha"] * x.to(F64) + p["gate"].to(F64) * p["beta_post"].to(F64))[4]
    assert bool(((r[4].to(F64) - want).abs() <= 4 * U * (x[4].abs() + 1).to(F64)).all())
    assert bool(torch.isfinite(r).all()) and bool(torch.isfinite(n).all())


def test_many_rows_a_cta_and_rows_behind_the_last_are_untouched():
    for T, H in ((9000, 64), (5003, 512), (2500, 1088), (1300, 7168)):
        x, y, p, dn, dr = _inputs(T + 1, H, F32, BF, "rms", "layer", True, True)
        big_r, big_n, big_s = torch.full_like(x, 7.0), torch.full_like(dn, 7.0), torch.full((T + 1, 4), 7.0, device=DEV)
        q = dict(p, gate_token=p["gate_token"][:T].contiguous())
        B.moe_residual_norm(x[:T], y[:T], q, big_r[:T], big_n[:T], big_s[:T])
        assert bool((big_r[T] == 7).all()) and bool((big_n[T] == 7).all()) and bool((big_s[T] == 7).all())
        _check_forward(x[:T], y[:T], q, big_r[:T], big_n[:T], big_s[:T])
        stats = _rounded_stats(y[:T], big_r[:T], q)
        dx, dy, grads = _backward(dn[:T], dr[:T], y[:T], big_r[:T], stats, q)
        rdx, rdy, ref = _reference(dn[:T], dr[:T], y[:T], big_r[:T], stats, q)
        assert _near(dx, *rdx) and _near(dy, *rdy)
        # (up to T rows a strand here: 8 of the bound's 62 roundings become T / 304 + 8)
        for k, g in grads.items():
            w, t = ref[k]
            assert _near(g, w, t * (T / 304 + 62) / 62), k


def test_empty_batch_graph_and_other_stream():
    H = 192
    x, y, p, dn, dr = _inputs(4, H, F32, F32, "layer", "rms", True, False)
    r, n, stats = _forward(x, y, p)
    dx, dy, grads = _backward(dn, dr, y, r, stats, p)
    e = {k: (v[:0] if torch.is_tensor(v) and k == "gate_token" else v) for k, v in p.items()}
    _, _, none = _backward(dn[:0], dr[:0], y[:0], r[:0], stats[:0], e)
    assert all(float(v.abs().sum()) == 0.0 for v in none.values())
    ws = torch.zeros(B.moe_residual_norm_backward_workspace_bytes(4, H), dtype=torch.uint8, device=DEV)
    r2, n2, s2 = torch.empty_like(r), torch.empty_like(n), torch.empty_like(stats)
    dx2, dy2, g2 = torch.empty_like(dx), torch.empty_like(dy), {k: torch.empty_like(v) for k, v in grads.items()}
    rb, rd, rg = _backward(dn, dr, y, r, s2.copy_(stats), p)

    def both(stream=None):
        B.moe_residual_norm(x, y, p, r2, n2, s2, stream=stream)
        B.moe_residual_norm_backward(dn, dr, y, r2, s2, p, dx2, dy2, g2, ws, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for go in (graph.replay, lambda: both(side)):
        for t in (r2, n2, s2, dx2, dy2, *g2.values()):
            t.fill_(float("nan"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        go()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(r2, r) and torch.equal(n2, n) and torch.equal(dx2, rb) and torch.equal(dy2, rd)
        assert all(torch.equal(g2[k], rg[k]) for k in rg)


def test_infinities_and_nan_stay_in_their_rows():
    x, y, p, dn, dr = _inputs(6, 576, BF, F32, "rms", "layer", True, False)
    y[2, 5], y[4, 7] = float("inf"), float("nan")
    r, n, stats = _forward(x, y, p)
    good = [0, 1, 3, 5]
    for t in (r, n, stats):
        assert bool(torch.isfinite(t[good]).all())
    assert bool(torch.isnan(r[4]).any()) and not bool(torch.isfinite(r[2]).all())


@pytest.mark.parametrize("kinds", [("rms", "layer", True, False, False), ("layer", "rms", True, True, True), ("none", "none", False, True, True)])
@pytest.mark.parametrize("T,H,xt,yt", [(9801, 1088, F32, F32), (9803, 576, F32, BF), (9901, 960, BF, F32), (9801, 1984, BF, BF), (4900, 2112, F32, BF), (5001, 4096, BF, F32),
                                       (2501, 7168, BF, BF), (2499, 7168, F32, F32), (2433, 8192, F32, F32), (700, 8192, BF, F32)])
def test_several_rows_a_cta(T, H, xt, yt, kinds):
    # batches long enough for CTAs that take several rows at a time, and for every stage of the rings
    x, y, p, dn, dr = _inputs(T, H, xt, yt, *kinds)
    r, n, stats = _forward(x, y, p)
    _check_forward(x, y, p, r, n, stats)
    stats = _rounded_stats(y, r, p)
    dx, dy, grads = _backward(dn, dr, y, r, stats, p)
    rdx, rdy, ref = _reference(dn, dr, y, r, stats, p)
    assert _near(dx, *rdx) and _near(dy, *rdy)
    # (up to T / 152 rows a strand: 8 of the bound's 62 roundings become T / 152 + 8)
    for k, g in grads.items():
        w, t = ref[k]
        assert _near(g, w, t * (T / 152 + 62) / 62), k


FIRST = """
import torch
from expert_routed_ffn_router_gb300 import binding as B
T, H, bf = 45, 256, torch.bfloat16
new = lambda *s, dtype=bf: torch.ones(*s, dtype=dtype, device="cuda")
one = torch.ones(H, device="cuda")
p = dict(post="layer", pre="rms", gamma_post=one, gamma_pre=one)
x, y, r, n, st = new(T, H), new(T, H), new(T, H), new(T, H), new(T, 4, dtype=torch.float32)
ws = torch.zeros(B.moe_residual_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
B.moe_residual_norm_backward(n, x, y, r, st, p, new(T, H), new(T, H), {}, ws)
B.moe_residual_norm(x, y, p, r, n, st)
torch.cuda.synchronize()
"""


def test_first_call_of_a_process():
    # its dynamic shared memory is exactly the 48 KB that need no attribute, beside static arrays
    subprocess.run([sys.executable, "-c", FIRST], check=True, timeout=300)
