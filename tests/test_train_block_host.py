"""The training block's host side (CPU: no kernel runs)."""
import pytest

from expert_routed_ffn_router_gb300 import binding as B
from expert_routed_ffn_router_gb300 import train


def test_fit_raises_with_the_condition_that_the_kernels_recorded(monkeypatch):
    words = [B.MOE_ERR_DEVICE_TIMEOUT]                # (reading the word resets it)

    class Block:
        grads = {}

        def __init__(self, *a, **k):
            pass

        def forward(self, x):
            return x

        def backward(self, dout):
            return dout, {}

        def status(self):
            return words.pop() if words else 0
    monkeypatch.setattr(train, "MoETrainBlock", Block)
    with pytest.raises(B.MoeError) as e:
        train.fit(steps=1, T=8, H=64, E=4, K=2, I=64, Is=0, device="cpu")
    assert e.value.status == B.MOE_ERR_DEVICE_TIMEOUT
