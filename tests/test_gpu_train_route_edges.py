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
