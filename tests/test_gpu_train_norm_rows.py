"""The layer norm's launches whose CTAs take several rows each, from a ring of shared-memory
stages: values, and waits on the ring that run out."""
import pytest
import torch

import test_gpu_train_norm as N
from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64 = N.DEV, N.BF, N.F32, N.F64


# Rows of a CTA: 9 or more in every case, more than twice the ring's four stages at most, and not
# the same number in every CTA (up to 512 columns backward, 2 to 9 rows a warp).  (The forward pass takes the ring from 8 rows a CTA on: 19456 rows
# of 1088, 10944 of 2112, 3648 of 7168, 2432 of 8256 and 1216 of 16384 with 152 SMs.)
FORWARD = [(22501, 1088), (12501, 2112), (4201, 7168), (2801, 8256), (1501, 16384)]
BACKWARD = [(6001, 64), (22001, 256), (7001, 512), (22501, 576), (11701, 1024), (9101, 2112), (4001, 7168),
            (1501, 8256), (1501, 16384)]


@pytest.mark.parametrize("T,H", FORWARD)
@pytest.mark.parametrize("xt", [BF, F32])
def test_forward_rows(T, H, xt):
    x, gamma, beta, _, _ = N._norm_inputs(T, H, xt, seed=8, offset=0.5)
    y, mean, rstd = N._forward(x, gamma, beta)
    X = x.to(F64)
    mu = X.mean(1, keepdim=True)
    r = ((X - mu).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    ref = gamma.to(F64) * (X - mu) * r + beta.to(F64)
    size = X.abs().amax(1, keepdim=True)
    assert bool(((mean.to(F64) - mu[:, 0]).abs() <= N.SUM * size[:, 0]).all())
    assert bool(((rstd.to(F64) / r[:, 0] - 1).abs() <= 2 * N.SUM * (1 + size[:, 0] * r[:, 0])).all())
    tol = 2.0 ** -8 * ref.abs() + 4 * N.SUM * (1 + size * r) * (gamma.to(F64).abs() * size * r + beta.to(F64).abs())
    assert bool(((y.to(F64) - ref).abs() <= tol).all())


@pytest.mark.parametrize("T,H", BACKWARD)
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("with_res", [False, True])
def test_backward_rows(T, H, xt, with_res):
    x, gamma, _, dy, res = N._norm_inputs(T, H, xt, seed=9)
    X = x.to(F64)
    mean = X.mean(1).float()
    rstd = ((X - X.mean(1, keepdim=True)).square().mean(1) + 1e-5).rsqrt().float()
    dx, dg, db = N._backward(dy, x, gamma, mean, rstd, res if with_res else None)
    D, G, r = dy.to(F64), gamma.to(F64), rstd.to(F64)[:, None]
    xh = (X - mean.to(F64)[:, None]) * r
    a = G * D
    ref = r * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    mag = r * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    if with_res:
        ref = ref + res.to(F64)
        mag = mag + res.to(F64).abs()
    step = 2.0 ** -8 if xt == BF else 2.0 ** -24
    assert bool(((dx.to(F64) - ref).abs() <= step * ref.abs() + 2 * N.SUM * mag).all())
    # a weight's sum: the rows of a CTA (or warp) one after the other, then the CTAs in 8 strands,
    # 10 CTAs an SM at most; a few roundings of each term
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tol = (T / sms + 10 * sms / 8 + 16) * 2.0 ** -24
    assert bool(((dg.to(F64) - (D * xh).sum(0)).abs() <= tol * (D * xh).abs().sum(0)).all())
    assert bool(((db.to(F64) - D.sum(0)).abs() <= tol * D.abs().sum(0)).all())


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
