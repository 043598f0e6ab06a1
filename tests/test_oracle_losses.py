"""The losses' oracle on the CPU: its gradients against differences, and values worked out by hand."""

import math

import numpy as np
import pytest

from oracle import losses


def _case(seed=0, rows=9, vocab=11):
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(rows, vocab)) * 2
    labels = rng.integers(0, vocab, rows)
    labels[[2, 5]] = -100
    seq_start = [0, 3, 3, 7, rows]  # the second sequence is empty
    now = losses.token_logp(logits, labels, 0.8)
    # ratios away from the clip's edges, on both sides of them
    ratio = np.array([0.5, 0.9, 1.0, 1.05, 1.6, 1.1, 0.7, 1.4, 0.95])
    return logits, labels, seq_start, now - np.log(ratio), now + rng.normal(size=rows) * 0.5, rng.normal(size=rows)


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("mean", ["token", "sequence"])
@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_against_differences(mean, kl):
    x, y, start, old, ref, adv = _case()
    kw = dict(ref=ref if kl else None, clip_low=0.2, clip_high=0.3, kl_coef=kl, temperature=0.8, mean=mean)
    got = losses.policy_loss(x, y, old, adv, start, **kw)
    want = _differences(lambda v: losses.policy_loss(v, y, old, adv, start, **kw)["stats"][0], x)
    # central differences at h = 1e-5: h^2 times a third derivative of order 1, and 1e-16 / h of rounding
    np.testing.assert_allclose(got["dlogits"], want, atol=1e-9)
    assert not got["dlogits"][[2, 5]].any()


@pytest.mark.parametrize("kw", [dict(form="sigmoid"), dict(form="sigmoid", label_smoothing=0.2),
                                dict(form="square", target=0.3), dict(form="square", length_normalized=True)])
def test_preference_gradient_against_differences(kw):
    x, y, start, _, ref, _ = _case(seed=3)
    kw = dict(kw, beta=0.7, temperature=0.8)
    got = losses.preference_loss(x, y, ref, start, **kw)
    want = _differences(lambda v: losses.preference_loss(v, y, ref, start, **kw)["stats"][0], x)
    np.testing.assert_allclose(got["dlogits"], want, atol=1e-9)


def test_values_by_hand():
    x = np.zeros((2, 4))
    assert np.allclose(losses.token_logp(x, [1, -1]), [-math.log(4), 0.0])
    # ratio 2 with a positive advantage is held at 1.2; with a negative one it is not
    lp = np.array([-1.0, -1.0])
    stats, slope = losses.policy_from_logp(lp, lp - math.log(2), np.array([3.0, -3.0]), np.array([0.5, 0.5]))
    assert np.allclose(stats, [0.5 * -3.6 + 0.5 * 6, 0.5 * -3.6 + 0.5 * 6, 0, 0.5])
    assert np.allclose(slope, [0.0, 3.0])
    # equal log ratios: log 2, and a slope of beta / 2 each way
    stats, ratios, slope = losses.preference_from_logp([-1, -2], [0, 0], [-1.5, -2.5], [0, 1, 2], beta=0.2)
    assert np.allclose(stats, [math.log(2), 0.1, 0.1, 0]) and np.allclose(slope, [-0.1, 0.1])


def test_nothing_labelled():
    x, y, start, old, ref, adv = _case()
    got = losses.policy_loss(x, np.full_like(y, -1), old, adv, start, ref=ref, kl_coef=0.1)
    assert not got["stats"].any() and not got["dlogits"].any()
