"""The entry points at the layer's edges as a training step uses them: the block with a norm and a
gate behind its experts, experts of the caller between dispatch and combine, and orthogonalised
updates.

Tolerances (2-norm of the difference over that of the result): a rounding to bf16 is at most 2^-8 of a
value; the counts of roundings are given at each test."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B
from expert_routed_ffn_router_gb300 import train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
STEP = 2.0 ** -8


def _rel(a, b):
    return float((a.to(F64) - b).norm() / b.norm())


def _norm(v, kind, eps):
    mu = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    return (v - mu) * ((v - mu).square().mean(1, keepdim=True) + eps) ** -0.5


@pytest.mark.parametrize("post,beta,gate,alpha", [("rms", False, True, 1.0), ("layer", True, False, 0.8), ("none", False, True, 1.0)])
@pytest.mark.parametrize("xt", [F32, BF])
@pytest.mark.parametrize("Is", [128, 0])
def test_block_with_a_norm_behind_its_experts(post, beta, gate, alpha, xt, Is):
    T, H, E, K, I = 70, 256, 16, 2, 128
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w = train.random_weights(H, E, I, Is, DEV, seed=4)
    w["gamma"] = 1 + 0.1 * r(H)
    if post != "none":
        w["gamma_post"] = 1 + 0.1 * r(H)
    if beta:
        w["beta_post"] = 0.1 * r(H)
    if gate:
        w["gate"] = 0.5 + 0.2 * r(H)
    block = train.MoETrainBlock(w, T, K, x_dtype=xt, post=post, alpha=alpha)
    x, dout = r(T, H).to(xt), r(T, H).to(xt)
    out = block.forward(x).clone()
    dx, grads = block.backward(dout)
    assert block.status() == 0
    # in 64 bits, at the values of n, the logits, the selection and Y that the forward pass left
    p = {k: v.to(F64).requires_grad_(True) for k, v in w.items()}
    X = x.to(F64).requires_grad_(True)
    n = p["gamma"] * _norm(X, "layer", block.eps) + p["beta"]
    n = n + (block.n.to(F64) - n).detach()
    idx = block.topk_idx.long()
    l = n @ p["W_gate"].t()
    l = l + (block.logits.to(F64) - l).detach()
    v = torch.sigmoid(l).gather(1, idx)
    v = v / v.sum(1, keepdim=True)
    ffn = lambda t, a, b, c: (torch.nn.functional.silu(t @ a) * (t @ b)) @ c
    Y = torch.zeros_like(X)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            Y = Y.index_add(0, t, v[t, j][:, None] * ffn(n[t], p["W1"][e], p["W3"][e], p["W2"][e]))
    if Is:
        Y = Y + ffn(n, p["W1s"], p["W3s"], p["W2s"])
    Y = Y + (block.Y.to(F64) - Y).detach()
    b = Y if post == "none" else p["gamma_post"] * _norm(Y, post, block.eps) + (p["beta_post"] if beta else 0.0)
    ref = alpha * X + (b * p["gate"] if gate else b)
    assert _rel(out, ref.detach()) <= (STEP if xt == BF else 1e-5)
    ref.backward(dout.to(F64))
    # the stream's part of dx is exact up to its rounding; the norm's inherits five roundings
    inner = X.grad - alpha * dout.to(F64)
    slack = float(dout.to(F64).norm()) * (2 * STEP if xt == BF else 1e-6)
    assert float((dx.to(F64) - X.grad).norm()) <= 5 * STEP * float(inner.norm()) + 2 * slack
    for name, got in grads.items():
        lim = 1e-5 if name in ("gamma_post", "beta_post", "gate") else 6 * STEP if name in ("gamma", "beta") else 3 * STEP
        assert _rel(got, p[name].grad) <= lim, name


def test_default_block_is_joined_as_before():
    w = train.random_weights(256, 8, 128, 128, DEV)
    x, dout = torch.randn(64, 256, device=DEV), torch.randn(64, 256, device=DEV)
    plain = train.MoETrainBlock(w, 64, 2)
    assert not plain.joined
    out, (dx, grads) = plain.forward(x).clone(), plain.backward(dout)
    assert torch.equal(out, x + plain.Y)
    one = train.MoETrainBlock(dict(w, gate=torch.ones(256, device=DEV)), 64, 2)
    assert torch.equal(one.forward(x), out)
    dx1, grads1 = one.backward(dout)
    assert torch.equal(dx1, dx) and all(torch.equal(grads1[k], grads[k]) for k in grads)


@pytest.mark.parametrize("graph", [False, True])
def test_experts_of_the_caller(graph):
    # dispatch -> the caller's experts (here a two-layer one with another activation) -> combine ->
    # joined stream and next norm, and back; the stream's and the slots' gradients in 64 bits
    T, H, E, K, D = 90, 320, 8, 3, 96
    g = torch.Generator(device=DEV).manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, X, w = r(T, H), r(T, H).to(BF), torch.rand(T, K, generator=g, device=DEV)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, 1).indices.to(I32)
    idx[5, 1] = -1                              # a pair that was rejected
    U, V = 0.05 * r(E, H, D), 0.1 * r(E, D, H)
    dn, dr = r(T, H).to(BF), r(T, H)
    p = dict(post="rms", pre="layer", alpha=0.9, gamma_post=1 + 0.1 * r(H), gate=0.5 + 0.1 * r(H), gamma_pre=1 + 0.1 * r(H),
             beta_pre=0.1 * r(H))
    new = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device=DEV)
    counts, off, perm, slot = new(E, dtype=I32), new(E + 1, dtype=I32), new(T * K, dtype=I32), new(T, K, dtype=I32)
    Xp, Yp, Y = new(T * K, H, dtype=BF), new(T * K, H, dtype=BF), new(T, H)
    s, n, st = new(T, H), new(T, H, dtype=BF), new(T, 4)
    dx, dY, dYp, dw = new(T, H), new(T, H, dtype=BF), new(T * K, H, dtype=BF), new(T, K)
    dXp, dX = new(T * K, H, dtype=BF), new(T, H)
    grads = {k: new(H) for k, v in p.items() if torch.is_tensor(v)}
    ws = torch.zeros(max(B.moe_workspace_bytes(T, H, E, K, 64, 0), B.moe_residual_norm_backward_workspace_bytes(T, H)),
                     dtype=torch.uint8, device=DEV)

    def experts(rows, of, dt):
        return (torch.tanh(rows.to(dt)[:, None] @ U.to(dt)[of]) @ V.to(dt)[of])[:, 0]

    def experts_back(rows, of, d, dt):
        t = torch.tanh(rows.to(dt)[:, None] @ U.to(dt)[of])
        return (((d.to(dt)[:, None] @ V.to(dt)[of].mT) * (1 - t * t)) @ U.to(dt)[of].mT)[:, 0]
    of = torch.zeros(T * K, dtype=torch.long, device=DEV)

    def step():
        B.moe_dispatch(X, idx, E, counts, off, perm, slot, Xp, None, ws)
        of.copy_(torch.searchsorted(off[1:].long(), torch.arange(T * K, device=DEV), right=True).clamp(max=E - 1))
        Yp.copy_(experts(Xp, of, F32))
        B.moe_combine(Yp, slot, w, None, Y)
        B.moe_residual_norm(x, Y, p, s, n, st)
        B.moe_residual_norm_backward(dn, dr, Y, s, st, p, dx, dY, grads, ws)
        B.moe_combine_backward(dY, Yp, slot, w, dYp, dw)
        dXp.copy_(experts_back(Xp, of, dYp, F32))
        B.moe_dispatch_backward(dXp, slot, None, dX)
    step()
    B.moe_read_status(ws)                       # (the rejected pair)
    if graph:
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        for t in (Yp, Y, s, n, st, dx, dY, dYp, dw, dXp, dX):
            t.zero_()
        gr.replay()
    live = slot >= 0
    assert int((~live).sum()) == 1 and float(dw[~live].abs().max()) == 0.0
    X64, w64, x64 = X.to(F64).requires_grad_(True), w.to(F64).requires_grad_(True), x.to(F64).requires_grad_(True)
    q = {k: v.to(F64).requires_grad_(True) if torch.is_tensor(v) else v for k, v in p.items()}
    y64 = torch.zeros(T, H, dtype=F64, device=DEV)
    for j in range(K):
        t = live[:, j].nonzero().squeeze(1)
        y64 = y64.index_add(0, t, w64[t, j][:, None] * experts(X64[t], idx[t, j].long(), F64))
    y64 = y64 + (Y.to(F64) - y64).detach()      # at the values that the forward pass left
    r64 = 0.9 * x64 + q["gate"] * q["gamma_post"] * _norm(y64, "rms", 1e-5)
    n64 = q["gamma_pre"] * _norm(r64, "layer", 1e-5) + q["beta_pre"]
    assert _rel(s, r64.detach()) <= 1e-5 and _rel(n, n64.detach()) <= STEP
    ((dn.to(F64) * n64).sum() + (dr.to(F64) * r64).sum()).backward()
    assert _rel(dx, x64.grad) <= 1e-5
    for k, v in grads.items():
        assert _rel(v, q[k].grad) <= 1e-5, k
    # dw: dY and the rows Yp are rounded; dX: dY, dYp and dXp
    assert _rel(dw, w64.grad) <= 2 * STEP and _rel(dX, X64.grad) <= 3 * STEP


def test_muon_step_and_fit():
    g = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w = dict(W1=(0.1 * r(6, 96, 64)).to(BF), W2s=(0.1 * r(64, 160)).to(BF))
    before = {k: v.to(F64) for k, v in w.items()}
    grads = dict(W1=r(6, 96, 64).to(BF), W2s=r(64, 160))
    opt = train.Muon(w, lr=0.05, decay=0.1, experts=4)
    parts = train.Muon({k: v.clone() for k, v in w.items()}, lr=0.05, decay=0.1)
    for _ in range(2):
        opt.step(grads)
        parts.step(grads)
    assert opt.status() == 0
    for k, v in grads.items():
        assert torch.equal(w[k], parts.weights[k]) and torch.equal(opt.master[k], parts.master[k])
        u, m, W = v.to(F64).view(-1, *v.shape[-2:]), 0, before[k].view(-1, *v.shape[-2:])
        for _ in range(2):
            m = 0.95 * m + u
            x = u + 0.95 * m
            x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
            for _ in range(5):
                A = x @ x.mT
                x = 3.4445 * x - 4.7750 * (A @ x) + 2.0315 * (A @ (A @ x))
            W = (1 - 0.05 * 0.1) * W - 0.05 * 0.2 * max(v.shape[-2:]) ** 0.5 * x
        # the update: its rounding and 6.2e-3 at most before it
        moved = W - before[k].view_as(W)
        assert float((opt.master[k].to(F64).view_as(W) - W).norm()) <= (6.2e-3 + STEP) * float(moved.norm())
        assert torch.equal(w[k], opt.master[k].to(BF))
    losses = train.fit(steps=3, T=64, muon=True)
    assert len(losses) == 3 and all(v == v for v in losses)


def test_tensors_of_another_device_are_refused(monkeypatch):
    # (the current device is said to be another one: nothing is launched)
    T, H, K = 4, 128, 2
    x, y = torch.zeros(T, H, device=DEV), torch.zeros(T * K, H, device=DEV, dtype=torch.bfloat16)
    slot = torch.arange(T * K, device=DEV, dtype=torch.int32).view(T, K)
    n, stats, ws = y[:T], torch.zeros(T, 4, device=DEV), torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    calls = [lambda: B.moe_combine_backward(x, y, slot, None, y),
             lambda: B.moe_dispatch_backward(y, slot, None, x),
             lambda: B.moe_residual_norm(x, x, {}, x),
             lambda: B.moe_residual_norm_backward(None, x, None, x, stats, {}, x, n, {}, ws),
             lambda: B.moe_orthogonalize(n, n, ws)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in (lambda: B.moe_orthogonalize(n, n, ws.cpu()), lambda: B.moe_dispatch_backward(y, slot.cpu(), None, x)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current one is 1"):
            call()
