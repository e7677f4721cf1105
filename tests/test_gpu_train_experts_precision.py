"""How near d topk_w of the expert FFN's backward pass comes to 64 bits at a depth of 7168, which
the sums continued in fp32 registers are for.

With positive operands every sum grows steadily, so that what the tensor core cuts off adds up.  A
sum of n MMAs (16 products each) loses 2^-23 of its partial sum an MMA at most, half the final
one on average: (n + 1) 2^-24 of it; its chunks (24 MMAs of bf16 rows, 32 of 8-bit rows) add up in
at most 19 roundings of 2^-24.  <p, h> carries that of p, u and g, the last 1 + g (1 - s) <= 1.28
fold, and 20 roundings of its own (sigmoid, products, the sum over I).  (Kernels with one sum over
all 448 MMAs measured 5 and 9e-5 here, where these bounds are 1e-5.)"""
import pytest

import test_gpu_train_experts as X
from expert_routed_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed,mmas,chunks", [(False, 24, 19), (True, 32, 14)])
def test_d_topk_w_of_long_sums(packed, mmas, chunks):
    T, H, E, K, I = 200, 7168, 4, 2, 256
    p = X._problem(T, H, E, K, I, packed, seed=3)
    x = p["xv"].abs()
    p["x"], p["xs"] = B.moe_checkpoint_pack(x) if packed else (x, None)
    p["xv"] = B.moe_checkpoint_unpack(p["x"], p["xs"]) if packed else x
    p["dY"] = p["dY"].abs()
    for n in ("W1", "W3", "W2"):                    # (g and u near 2)
        p[n] = (p[n].abs() / 90).to(X.BF)
    o, ws = X.backward(p)
    assert B.moe_read_status(ws) == 0
    ref, _ = X.reference(p)
    off = (o["dw"].to(X.F64) / ref["dw"] - 1).abs().max()
    assert float(off) <= (3.28 * (mmas + 1 + chunks) + 20) * 2.0 ** -24, float(off)
