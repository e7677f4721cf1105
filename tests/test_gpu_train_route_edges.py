"""Routing from given logits where sums cancel, underflow or saturate: the selection has to be
the definition's in 64 bits, weights and gradients right relative to their own size."""
import numpy as np
import pytest
import torch

import test_gpu_train_route as R
from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = R.DEV
F32 = torch.float32


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1e4, 1e5])
def test_group_sums_that_cancel(scoring, size):
    # one expert of each group with bias +size, the others -size (and a spread of 0.2): a group's
    # two largest values cancel in their sum, their roundings (2^-24 size) do not
    T, E = 20000, 256
    rng = np.random.default_rng(0)
    b = (0.2 * rng.random(E)).astype(np.float32) - np.float32(size)
    for g in range(8):
        b[g * 32 + int(rng.integers(32))] += np.float32(2 * size)
    R._check(R._logits(T, E, F32, seed=11), torch.from_numpy(b).to(DEV), 8, scoring=scoring, n_group=8, topk_group=4,
             group_top=2)


@pytest.mark.parametrize("E,group_top", [(16, 2), (256, 2), (256, 1)])
def test_groups_of_masked_and_of_excluded_experts(E, group_top):
    # group 0 holds experts with a bias of -inf, group 1 one unmasked expert and masked ones: the
    # order of the two does not depend on how many experts there are
    l = torch.full((3, E), -float("inf"), device=DEV)
    l[:, :E // 2] = 0.25
    l[:, E // 2 + 5] = torch.tensor([0.5, -3.0, 20.0], device=DEV)
    b = torch.zeros(E, device=DEV)
    b[:E // 2] = -float("inf")
    for scoring in ("sigmoid", "softmax"):
        idx, _ = R._check(l, b, 8, scoring=scoring, n_group=2, topk_group=1, group_top=group_top)
        assert bool((idx[:, 0] == E // 2 + 5).all())


# A weight is a score over a sum of K scores: each a handful of fp32 roundings (exp, its
# argument's rounding of up to 128 x 2^-24, sum, reciprocal).
REL = (128 + 32) * 2.0 ** -24


def _selected_weights(l, idx):
    """softmax of the selected logits, 64 bits."""
    v = np.take_along_axis(l.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64), 1)
    e = np.exp(v - v.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


@pytest.mark.parametrize("depth", [95.0, 120.0])
def test_softmax_weights_of_experts_far_below_the_maximum(depth):
    # a bias that keeps the row's largest logits out: the weights are a softmax of the selected
    T, E, K = 64, 40, 6
    l = R._logits(T, E, F32, seed=12)
    l[:, 3] = l[:, 3] + depth
    b = torch.zeros(E, device=DEV)
    b[3] = -10.0
    l[1, 7] = -float("inf")
    idx, w = R._route(l, b, K, scoring="softmax")
    assert not bool((idx == 3).any())
    ref = _selected_weights(l, idx)
    assert bool((np.abs(w.double().cpu().numpy() - ref) <= REL * ref).all())
    # ... and the gradient is that of these weights
    dw = torch.linspace(-1, 1, K, device=DEV).expand(T, K).contiguous()
    out = torch.empty_like(l)
    B.moe_route_logits_backward(l, dict(scoring="softmax"), idx, dw, out)
    d = dw.double().cpu().numpy()
    want = ref * (d - (ref * d).sum(1, keepdims=True))
    got = out.gather(1, idx.long()).double().cpu().numpy()
    assert bool((np.abs(got - want) <= 4 * REL * ref).all())


@pytest.mark.parametrize("at", [-60.0, -90.0, -300.0])
def test_sigmoid_weights_of_small_scores(at):
    # scores that fp32 cannot hold, whose ratios it can: sigmoid(l) is e^l to e^l of itself
    T, E, K = 64, 40, 6
    l = R._logits(T, E, F32, seed=13) + at
    l[1, :20] = -float("inf")
    l[2] = -float("inf")
    l[3] = -1e35                                    # a score of 0 in 64 bits too
    idx, w = R._route(l, None, K)
    live = [t for t in range(T) if t not in (2, 3)]
    ref = _selected_weights(l[live], idx[live])
    assert bool((np.abs(w[live].double().cpu().numpy() - ref) <= REL * ref).all())
    assert not bool(w[[2, 3]].any())
    dw = torch.linspace(-1, 1, K, device=DEV).expand(T, K).contiguous()
    out = torch.empty_like(l)
    B.moe_route_logits_backward(l, None, idx, dw, out)
    d = dw[live].double().cpu().numpy()
    want = ref * (d - (ref * d).sum(1, keepdims=True))
    got = out.gather(1, idx.long())[live].double().cpu().numpy()
    assert bool((np.abs(got - want) <= 4 * REL * ref).all())
    assert not bool(out[[2, 3]].any())


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_saturated_gates(renorm):
    # 1 - s of a logit of 10 to 80 is e^-l: relative to its size
    T, E = 71, 8
    l = torch.full((T, E), -5.0, device=DEV)
    l[:, 2] = torch.arange(10, 81, device=DEV).float()
    l[:, 5] = torch.arange(10, 81, device=DEV).float() + 0.5
    idx = torch.tensor([[5, 2]], dtype=torch.int32, device=DEV).expand(T, 2).contiguous()
    dw = torch.tensor([[1.0, -0.5]], device=DEV).expand(T, 2).contiguous()
    out = torch.empty_like(l)
    B.moe_route_logits_backward(l, dict(renorm=renorm), idx, dw, out)
    x = l.double().cpu().gather(1, idx.long().cpu()).numpy()
    s, q, d = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x)), dw.double().cpu().numpy()
    w = s / s.sum(1, keepdims=True)
    want = w * (d - (w * d).sum(1, keepdims=True)) * q if renorm else s * q * d
    got = out.gather(1, idx.long()).double().cpu().numpy()
    assert bool((np.abs(got - want) <= REL * np.abs(want)).all())
    out[:, [2, 5]] = 0
    assert not bool(out.any())
