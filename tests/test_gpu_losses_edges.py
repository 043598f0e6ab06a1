"""The losses on a GB300 where parts of them are infinite, not a number, or multiplied by nothing."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# (rows, vocab, type): a few rows, more than a few, a cluster a row, streamed rows in clusters of 1 and 2
SIZES = [(20, 60, torch.float32), (24, 61, torch.bfloat16), (600, 60, torch.float32), (24, 32000, torch.float32),
         (640, 16500, torch.bfloat16), (640, 20003, torch.float32)]


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def normal(rows, vocab, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 2).to(dtype)
    return x, torch.randint(0, vocab, (rows,), generator=gen, device="cuda")


@pytest.mark.parametrize("rows,vocab,dtype", SIZES)
def test_rows_outside_the_sequences(g, rows, vocab, dtype):
    """Labelled rows of no sequence have no gradient, whatever they hold."""
    x, labels = normal(rows, vocab, dtype)
    x[:, 3::7] = -float("inf")
    labels = torch.where(labels % 7 == 3, labels - 1, labels)
    x[0], x[1, 2], x[2] = float("nan"), float("inf"), -float("inf")
    x[rows - 1, vocab - 1] = float("nan")
    start = torch.tensor([3, 7, 7, 11, rows - 2], device="cuda")
    old = torch.nan_to_num(g.ar_token_logp(x, labels)) - 0.1
    for call in (lambda **kw: g.ar_policy_loss(x, labels, old, torch.ones_like(old), start, **kw),
                 lambda **kw: g.ar_policy_loss(x, labels, old, torch.ones_like(old), start, reduction="sequence", **kw),
                 lambda **kw: g.ar_preference_loss(x, labels, old, start, **kw)):
        stats, *_, d = call()
        assert torch.isfinite(stats).all() and torch.isfinite(d).all()
        assert not d[:3].any() and not d[rows - 2:].any() and d[3:rows - 2].any()


@pytest.mark.parametrize("rows,vocab,dtype", SIZES)
def test_divergence_that_is_only_reported(g, rows, vocab, dtype):
    """With a coefficient of 0 the KL term is a statistic: where it leaves fp32's range, loss and gradient stay."""
    x, labels = normal(rows, vocab, dtype)
    at = torch.arange(rows, device="cuda")
    x[at[:5], labels[:5]] = -200.0
    x[at[5:7], labels[5:7]] = -float("inf")
    adv = torch.where(at % 2 == 0, 1.0, -0.5)
    old = torch.full((rows,), -5.0, device="cuda")
    ref = torch.full((rows,), -1.0, device="cuda")
    start = torch.tensor([0, rows // 2, rows], device="cuda")
    want = g.ar_policy_loss(x, labels, old, adv, start)
    got = g.ar_policy_loss(x, labels, old, adv, start, ref_logp=ref)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[2]).all()
    assert torch.equal(got[0][[0, 1, 3]], want[0][[0, 1, 3]]) and float(got[0][2]) == math.inf
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("rows,vocab,dtype", SIZES)
def test_tokens_without_advantage(g, rows, vocab, dtype):
    """An advantage of 0 has no surrogate and no slope, however far the ratio is from 1."""
    x, labels = normal(rows, vocab, dtype)
    at = torch.arange(rows, device="cuda")
    lp = g.ar_token_logp(x, labels)
    old = torch.where(at % 3 == 0, lp - 150.0, lp)  # ratios beyond fp32's range
    adv = torch.where(at % 3 == 0, 0.0, 1.0)
    stats, _, d = g.ar_policy_loss(x, labels, old, adv)
    n = int((at % 3 != 0).sum())
    assert abs(float(stats[0]) + n / rows) < 1e-4 and float(stats[0]) == float(stats[1]) and float(stats[3]) == 0.0
    assert not d[at % 3 == 0].any() and torch.isfinite(d).all() and d[1].any()
    # with an advantage such a ratio is held by the clip, or makes the loss infinite
    stats, _, d = g.ar_policy_loss(x, labels, old, torch.ones_like(old), clip_high=0.25)
    assert abs(float(stats[0]) + (n + 1.25 * (rows - n)) / rows) < 1e-4
    assert not d[at % 3 == 0].any() and torch.isfinite(d).all()
    assert float(g.ar_policy_loss(x, labels, old, -torch.ones_like(old))[0][0]) == math.inf


@pytest.mark.parametrize("rows,vocab,dtype", SIZES)
def test_rejected_answers_that_are_ruled_out(g, rows, vocab, dtype):
    """-log sigmoid(z) at z = +inf is 0: a rejected answer of probability 0 adds nothing without smoothing."""
    x, labels = normal(rows, vocab, dtype)
    at = torch.arange(rows, device="cuda")
    start = torch.tensor([0, 5, 10, 13, rows], device="cuda")
    lp = g.ar_token_logp(x, labels)
    clean = g.ar_preference_loss(x, labels, lp, start, denominator=2.0)
    x[at[7], labels[7]] = -float("inf")
    stats, ratios, _, d = g.ar_preference_loss(x, labels, lp, start, denominator=2.0)
    # the other pair has ratios of 0, or rounding: half of log 2
    assert abs(float(clean[0][0]) - math.log(2)) < 1e-2 and abs(float(stats[0]) - math.log(2) / 2) < 1e-2
    assert float(ratios[1]) == -math.inf and float(stats[2]) == -math.inf and float(stats[3]) >= 0.5
    assert not d[:10].any() and torch.equal(d[10:], clean[3][10:])
    # the other way round the loss has no bound, and the slope is the steepest
    x[at[2], labels[2]] = -float("inf")
    x[at[7], labels[7]] = 0.0
    stats, ratios, _, d = g.ar_preference_loss(x, labels, lp, start, denominator=2.0, beta=0.5)
    assert float(stats[0]) == math.inf and float(ratios[0]) == -math.inf and torch.isfinite(d).all()
    assert abs(float(d[2, labels[2]]) + 0.25) < 1e-3 and abs(float(d[7].float().clamp(min=0).sum())) < 0.26
