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


def test_rows_are_kept_in_8_bits_only_where_asked_for():
    w = train.random_weights(64, 4, 64, 0, "cpu")
    assert train.MoETrainBlock(w, 8, 2).q is None
    assert train.MoETrainBlock(w, 8, 2, packed=False).q is None
    q = train.MoETrainBlock(w, 8, 2, packed=True).q
    assert q.shape == (8, 64) and q.element_size() == 1


@pytest.mark.parametrize("args,packed", [([], False), (["--bf16-rows"], False), (["--packed"], True)])
def test_the_commands_rows(monkeypatch, args, packed):
    seen = {}
    monkeypatch.setattr(train, "fit", lambda **k: seen.update(k) or [])
    train.main(args)
    assert seen["packed"] is packed
