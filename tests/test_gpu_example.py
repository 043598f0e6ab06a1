"""The post-training example: the operators together, as a program uses them."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("objective", ["policy", "preference"])
def test_rewards_rise(objective):
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g
    from examples.post_training import train

    rewards = train(objective, steps=10, ranks=2, answers=32, length=16, vocab=256, hidden=64)
    # answers start near one half by symmetry; the step's direction raises them
    assert abs(rewards[0] - 0.5) < 0.15 and sum(rewards[-3:]) / 3 > rewards[0] + 0.1, rewards
    assert g.ar_device_status() == g.AR_OK
