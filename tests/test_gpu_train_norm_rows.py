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


# (1 ns and copies: some waits run out, copies are in flight; 1 ms without copies: all run out)
@pytest.mark.parametrize("limit,stall", [(1, 0), (1_000_000, 1)])
@pytest.mark.parametrize("T,H,xt", [(22501, 1088, BF), (4001, 7168, F32), (4001, 7168, BF), (1301, 16384, F32)])
def test_forward_holds_where_waits_run_out(T, H, xt, limit, stall):
    x, gamma, beta, _, _ = N._norm_inputs(T, H, xt, seed=6)
    want = N._forward(x, gamma, beta)
    B.moe_debug_set_wait_limit(limit, stall)
    try:
        got = N._forward(x, gamma, beta)
        torch.cuda.synchronize()
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    # the same sums in another order: y within a step of bf16, and a few of fp32
    assert bool((got[1] - want[1]).abs().max() <= N.SUM * float(x.float().abs().max()))
    assert bool(((got[2] / want[2] - 1).abs() <= 1e-5).all())
    step = 2.0 ** -7 * want[0].to(F64).abs()
    assert bool(((got[0].to(F64) - want[0].to(F64)).abs() <= step + 1e-4).all())


def test_backward_without_its_copies_says_so():
    T, H = 400, 7168
    x, gamma, _, dy, res = N._norm_inputs(T, H, F32, seed=7)
    _, mean, rstd = N._forward(x, gamma, None)
    want = N._backward(dy, x, gamma, mean, rstd, res)
    ws = torch.zeros(B.moe_layer_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(t) for t in want]
    run = lambda: B.moe_layer_norm_backward(dy, x, gamma, mean, rstd, res, *out, ws)
    B.moe_debug_set_wait_limit(1_000_000, 1)
    try:
        run()
        assert B.moe_read_status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_set_wait_limit(0, 0)
    run()
    assert B.moe_read_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(out, want))
