"""The optimiser's chunks of a tensor's matrices on the GPU.

Tolerances.  out is the same matrices' result of one call, up to the order in which long sums are formed:
its fp32 sums may differ in their last bits, and with them a rounding to bf16 (2^-7 of a value between two
neighbours) here and there; the operands' roundings to fp16 (2^-10 between neighbours) flip likewise and
reach the result with the factors that the updates' own error has, below 6.2e-3 in 2-norm."""
import pytest
import torch

from expert_routed_ffn_router_gb300 import train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.mark.parametrize("shape,experts", [((3, 512, 2048), 2), ((7, 256, 2048), 4), ((9, 2100, 200), 5)])
def test_the_last_call_has_fewer_matrices(shape, experts):
    g = torch.Generator(device=DEV).manual_seed(6)
    w = (0.05 * torch.randn(shape, generator=g, device=DEV)).to(BF)
    grads = [torch.randn(shape, generator=g, device=DEV) for _ in range(2)]
    opt, whole = train.Muon({"W": w.clone()}, experts=experts), train.Muon({"W": w.clone()})
    m = torch.zeros(shape, device=DEV)
    for d in grads:
        opt.step({"W": d})
        whole.step({"W": d})
        m = torch.addcmul(d, m, torch.full_like(m, opt.mu))
    assert opt.status() == 0 and whole.status() == 0
    # every matrix's momentum is advanced once a step: one rounding of the fused product and sum, twice
    assert float((opt.momentum["W"] - m).abs().max()) <= 2.0 ** -22 * float(m.abs().max())
    assert torch.equal(opt.momentum["W"], whole.momentum["W"])
    a, b = opt.update["W"].to(F64), whole.update["W"].to(F64)
    off = torch.linalg.vector_norm(a - b, dim=(1, 2)) / torch.linalg.vector_norm(b, dim=(1, 2))
    assert float(off.max()) <= 6.2e-3 + 2.0 ** -7
