"""The layer norm's launches whose CTAs take several rows each, from a ring of shared-memory
stages: values, and waits on the ring that run out."""
import pytest
import torch

import test_gpu_train_norm as N
from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64 = N.DEV, N.BF, N.F32, N.F64


@pytest.mark.parametrize("H,xt", [(1024, F32), (7168, F32), (7168, BF), (16384, F32)])
def test_backward_waits_cut_short_end_with_a_status(H, xt):
    # a limit that copies in flight do not meet: the call ends, says so, and the next one is right
    T = 1700
    x, gamma, _, dy, res = N._norm_inputs(T, H, xt, seed=5)
    _, mean, rstd = N._forward(x, gamma, None)
    want = N._backward(dy, x, gamma, mean, rstd, res)
    out = [torch.empty_like(t) for t in want]
    ws = torch.zeros(B.moe_layer_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    run = lambda: B.moe_layer_norm_backward(dy, x, gamma, mean, rstd, res, *out, ws)
    B.moe_debug_set_wait_limit(1, 0)
    try:
        run()
        status = B.moe_read_status(ws)
        assert status in (0, B.MOE_ERR_DEVICE_TIMEOUT)
        if status == 0:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    run()
    assert B.moe_read_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(out, want))
