"""The host side of the orthogonalised updates: workspace sizes and the optimiser that chunks a tensor's
matrices (CPU: no kernel runs)."""
import os
import subprocess
import sys

import pytest
import torch

from expert_routed_ffn_router_gb300 import binding as B
from expert_routed_ffn_router_gb300 import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(64, 96), (128, 3000), (128, 3100), (300, 520), (7168, 100), (100, 7168), (2112, 1088), (512, 2048), (1, 32768),
          (32768, 32768)]


def test_workspace_of_no_matrices():
    # (in a process of its own: the division by the number of matrices ended it)
    code = ("from expert_routed_ffn_router_gb300 import binding as B\n"
            f"for s in {SHAPES!r}: assert 0 < B.moe_orthogonalize_workspace_bytes(0, *s) <= 4096, s\n")
    assert subprocess.run([sys.executable, "-c", code], timeout=300, cwd=ROOT).returncode == 0


def test_workspace_of_matrices_that_stay_on_the_chip():
    # up to 128 on the smaller side and 8 x 384 on the larger, all steps run in shared and tensor memory
    for b, r, c in ((256, 128, 3000), (65535, 128, 128), (1, 1, 1), (3, 3071, 127), (700, 24, 17)):
        assert 0 < B.moe_orthogonalize_workspace_bytes(b, r, c) <= 4096
    for r, c in ((129, 130), (128, 3073), (3073, 1), (300, 520)):
        assert B.moe_orthogonalize_workspace_bytes(2, r, c) > 2 * 6 * r * c


def _calls(monkeypatch):
    """Every call's matrices, bytes of workspace and addresses, in place of the kernels."""
    seen = []

    def call(g, out, ws, momentum=None, **k):
        out.fill_(1.0)
        momentum.add_(g)
        seen.append((g.shape, ws.numel(), [t.data_ptr() for t in (g, out, momentum)]))
    monkeypatch.setattr(B, "moe_orthogonalize", call)
    return seen


# (fewer matrices may need more: their sums are formed in parts)
@pytest.mark.parametrize("shape,experts", [((3, 512, 2048), 2), ((7, 256, 2048), 4), ((9, 200, 2100), 5), ((5, 64, 96), 2),
                                           ((512, 2048), 1), ((4, 300, 520), None)])
def test_muon_has_the_workspace_of_its_last_call_too(monkeypatch, shape, experts):
    w = torch.zeros(shape, dtype=torch.bfloat16)
    opt = train.Muon({"W": w}, experts=experts)
    seen = _calls(monkeypatch)
    opt.step({"W": torch.ones_like(w)})
    assert sum(s[0] for s, _, _ in seen) == (shape[0] if len(shape) == 3 else 1)
    for s, have, _ in seen:
        assert have >= B.moe_orthogonalize_workspace_bytes(*s), s


def test_muon_refuses_numbers_of_matrices_that_it_cannot_take(monkeypatch):
    w = torch.zeros(6, 64, 96, dtype=torch.bfloat16)
    for bad in (0, -1, -4, 1.5, "2"):      # (-1 took no step at all, 0 all matrices)
        with pytest.raises(ValueError, match="experts"):
            train.Muon({"W": w}, experts=bad)


# bf16 matrices of 35, 12 and 4 entries: 8, 2 and 2 of them end on a boundary of 16 bytes
@pytest.mark.parametrize("shape,experts,sizes", [((20, 5, 7), 9, [8, 8, 4]), ((5, 3, 4), 3, [2, 2, 1]), ((9, 2, 2), 2, [2] * 4 + [1]),
                                                 ((3, 5, 7), 8, [3]), ((3, 5, 7), None, [3]), ((5, 64, 96), 2, [2, 2, 1])])
def test_muon_takes_matrices_from_aligned_addresses_on(monkeypatch, shape, experts, sizes):
    w = torch.zeros(shape, dtype=torch.bfloat16)
    opt = train.Muon({"W": w}, experts=experts)
    seen = _calls(monkeypatch)
    opt.step({"W": torch.ones_like(w)})
    assert [s[0] for s, _, _ in seen] == sizes
    for s, have, at in seen:
        assert all(a % 16 == 0 for a in at) and have >= B.moe_orthogonalize_workspace_bytes(*s)
    assert bool((opt.momentum["W"] == 1).all())


@pytest.mark.parametrize("shape,experts", [((3, 5, 7), 2), ((20, 5, 7), 7), ((5, 3, 4), 1), ((2, 1, 1), 1)])
def test_muon_refuses_chunks_between_boundaries(shape, experts):
    # (refused by the second call of a step, after the first one's momentum, before)
    with pytest.raises(ValueError, match="experts"):
        train.Muon({"W": torch.zeros(shape, dtype=torch.bfloat16)}, experts=experts)
