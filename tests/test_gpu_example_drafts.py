"""The post-training example with drafted rollouts, clipped gradients and AdamW: it runs, and what it hands from one
operator to the next is what the next one expects."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


@pytest.mark.parametrize("objective", ["policy", "preference"])
@pytest.mark.parametrize("options", [dict(drafts=3), dict(max_norm=0.01), dict(drafts=2, max_norm=0.01, adamw=True)])
def test_runs(g, objective, options):
    from examples.post_training import train

    rewards = train(objective, steps=3, ranks=2, answers=16, length=8, vocab=128, hidden=32, **options)
    assert len(rewards) == 3 and all(0.0 <= r <= 1.0 for r in rewards)
    assert g.ar_device_status() == g.AR_OK


@pytest.mark.parametrize("drafts", [1, 2, 5])
def test_drafted_rollouts(g, drafts):
    """Chains of tokens (each before-token is the after-token of the place before), of the lengths asked for, with the
    log-probabilities of the policy that verified them."""
    from examples.post_training import Policy, drafted_rollouts

    policy, draft = Policy(200, 32, 0), Policy(200, 32, 1)
    gen = torch.Generator(device="cuda").manual_seed(5)
    before, after, start, logp = drafted_rollouts(policy, draft, 40, 12, 200, gen, drafts)
    lengths = start[1:] - start[:-1]
    assert ((lengths >= 1) & (lengths <= 12)).all() and start[-1] == len(before) == len(after) == len(logp)
    inner = torch.ones(len(before), dtype=torch.bool, device="cuda")
    inner[start[:-1]] = False
    assert torch.equal(before[inner], after[:-1][inner[1:]])
    assert ((after >= 0) & (after < 200)).all()
    want = torch.log_softmax(policy.logits(before).double(), 1).gather(1, after[:, None])[:, 0]
    # the logits come from fp32 products of other sizes (64 terms, scores of some units): 2^-24 a term at most
    assert (want - logp).abs().max() < 64 * 4 * 2.0 ** -23


def test_drafted_rollouts_have_the_policys_distribution(g):
    """The first tokens of many drafted answers: shares as the policy's, within 5 standard deviations."""
    from examples.post_training import Policy, drafted_rollouts

    policy, draft = Policy(12, 16, 0), Policy(12, 16, 1)
    gen = torch.Generator(device="cuda").manual_seed(6)
    before, after, start, _ = drafted_rollouts(policy, draft, 60000, 3, 12, gen, 2)
    p = torch.softmax(policy.logits(torch.arange(12, device="cuda")).double(), 1)
    for places in (start[:-1], torch.nonzero(torch.ones_like(before))[:, 0]):
        b, a = before[places], after[places]
        n = torch.bincount(b, minlength=12).double()
        share = torch.bincount(b * 12 + a, minlength=144).reshape(12, 12).double() / n[:, None]
        assert ((share - p).abs() <= 5 * (p * (1 - p) / n[:, None]).sqrt() + 1e-9).all()
