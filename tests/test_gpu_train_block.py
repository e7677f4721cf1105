"""The training block (train.MoETrainBlock): the entry points together, against automatic
differentiation of the block in 64 bits at the selection the GPU made.

Tolerances (2-norm of the difference over that of the result).  A rounding to bf16 is at most
2^-8 of a value.  Weight gradients carry three (dY, dg or du or hw, the result), the experts'
part of dx five (dY, dg and du, dX, the sum of the branches; the shared expert's dX), the gate's
gradient one (dY) and the fp32 sums after it."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B
from expert_routed_ffn_router_gb300 import train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64 = torch.float64
STEP = 2.0 ** -8


def _rel(a, b):
    return float((a.to(F64) - b).norm() / b.norm())


def _reference(block, x, dout, routing):
    """The block in 64 bits: the norm's output rounded to bf16 for the experts and the gate (and,
    packed, kept in 8 bits for the backward pass), as the block does."""
    w = {k: (None if v is None else v.to(F64).requires_grad_(True)) for k, v in block.w.items()}
    X = x.to(F64).requires_grad_(True)
    mu = X.mean(1, keepdim=True)
    n = w["gamma"] * (X - mu) * ((X - mu).square().mean(1, keepdim=True) + block.eps) ** -0.5 + w["beta"]
    kept = B.moe_checkpoint_unpack(block.q, block.scale) if block.packed else block.n
    n = n + (kept.to(F64) - n).detach()          # the kept values, the norm's gradient
    idx = block.topk_idx.long()
    l = n @ w["W_gate"].t()
    l = l + (block.logits.to(F64) - l).detach()  # the forward pass's logits, the kept rows' gradient
    s = torch.softmax(l, 1) if routing.get("scoring") == "softmax" else torch.sigmoid(l)
    v = s.gather(1, idx)
    if routing.get("renorm", True):
        v = v / v.sum(1, keepdim=True)
    ffn = lambda t, a, b, c: (torch.nn.functional.silu(t @ a) * (t @ b)) @ c
    Y = torch.zeros_like(X)
    for e in range(block.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            Y = Y.index_add(0, t, v[t, j][:, None] * ffn(n[t], w["W1"][e], w["W3"][e], w["W2"][e]))
    if block.shared:
        Y = Y + ffn(n, w["W1s"], w["W3s"], w["W2s"])
    (X + Y).backward(dout.to(F64))
    return (X + Y).detach(), X.grad, {k: w[k].grad for k in block.grads}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,E,K,I,Is,routing", [
    (70, 256, 16, 2, 128, 128, dict()),
    (33, 320, 8, 3, 192, 0, dict(scoring="softmax", renorm=False)),
    (200, 512, 32, 4, 128, 256, dict(n_group=8, topk_group=4, group_top=2)),
])
def test_step_against_automatic_differentiation(T, H, E, K, I, Is, routing, xt, packed):
    g = torch.Generator(device=DEV).manual_seed(T)
    w = train.random_weights(H, E, I, Is, DEV, seed=T)
    w["gamma"] = 1 + 0.1 * torch.randn(H, generator=g, device=DEV)
    w["beta"] = 0.1 * torch.randn(H, generator=g, device=DEV)
    block = train.MoETrainBlock(w, T, K, routing=routing or None, packed=packed, x_dtype=xt)
    x = torch.randn(T, H, generator=g, device=DEV).to(xt)
    dout = torch.randn(T, H, generator=g, device=DEV).to(xt)
    out = block.forward(x).clone()
    dx, grads = block.backward(dout)
    assert block.status() == 0
    ref_out, ref_dx, ref = _reference(block, x, dout, routing)
    # (forward on bf16 rows; the packed reference's are rounded to 4 bits besides: 2^-4)
    assert _rel(out, ref_out) <= (2 ** -4 if packed else 4 * STEP)
    inner = ref_dx - dout.to(F64)                # what goes through the norm
    slack = float(dout.to(F64).norm()) * (STEP if xt == torch.bfloat16 else 0.0)
    assert float((dx.to(F64) - dout.to(F64) - inner).norm()) <= 5 * STEP * float(inner.norm()) + 2 * slack
    for name in grads:
        lim = 6 * STEP if name in ("gamma", "beta") else 3 * STEP
        assert _rel(grads[name], ref[name]) <= lim, (name, _rel(grads[name], ref[name]))


def test_step_replays_in_a_graph():
    w = train.random_weights(256, 8, 128, 128, DEV)
    block = train.MoETrainBlock(w, 64, 2)
    x = torch.randn(64, 256, device=DEV)
    dout = torch.randn(64, 256, device=DEV)

    def step():
        block.forward(x)
        return block.backward(dout)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):                   # (first calls outside the capture)
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx, grads = step()
    x.mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    got = [dx.clone()] + [v.clone() for v in grads.values()]
    dx, grads = step()
    assert all(torch.equal(a, b) for a, b in zip(got, [dx] + list(grads.values())))


@pytest.mark.parametrize("packed", [True, False])
def test_fit_lowers_the_loss(packed):
    losses = train.fit(steps=40, T=256, packed=packed)
    assert losses[-1] < 0.8 * losses[0], (losses[0], losses[-1])


def test_backward_needs_a_forward():
    block = train.MoETrainBlock(train.random_weights(64, 4, 64, 0, DEV), 8, 2)
    with pytest.raises(RuntimeError, match="before forward"):
        block.backward(torch.zeros(8, 64, device=DEV))
