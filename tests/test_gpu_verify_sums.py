"""Sums over rows whose scores lie far apart: log-probabilities stay within what terms and sums may be off by."""

import numpy as np
import pytest
import torch

from oracle import verify as V

pytestmark = pytest.mark.gpu

# A term is the fp32 exponential of a number of magnitude below 32, rounded to 2^-20 of 1 (0.7 of that of the term), and
# is off by 2^-22 itself: below 2^-20. Below 128 it is four times the rounding, 2^-18.4 and 2^-22: below 2^-18. A sum may be
# off by 2^-20 more; the log-probability's own rounding is 2^-24 of it, and as much for its last steps.
NEAR, FAR, SUM = 2.0 ** -20, 2.0 ** -18, 2.0 ** -20
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def drawn_logp(g, row, token, temperature=1.0):
    """A token's log-probability from a call that verifies it as a draft that stands."""
    target = torch.stack([row, row]).cuda()
    u = torch.zeros(2).cuda()
    accepted, tokens, logp = g.ar_verify_drafts(target, torch.tensor([token]).cuda(), u, temperature=temperature)
    assert accepted.tolist() == [1] and tokens[0].item() == token
    return logp[0].item()


def check(g, row, token, room=NEAR + SUM):
    want = float(np.log(V.softmax(row.double().numpy())[token]))
    got = drawn_logp(g, row, token)
    assert abs(got - want) <= room + 2.0 ** -23 * abs(want), (got, want)


@pytest.mark.parametrize("level", [4194304.0, -4194304.0])
def test_many_far_scores_of_uneven_size(g, level):
    """Scores so large that their product with log2 e has no fraction, their maximum taken off first: of 32 tokens that
    lead their groups and 131040 others with a share of 2e-9 each, the others count 8e-6 together."""
    vocab = 131072
    row = torch.full((vocab,), level - 20.0)
    row[torch.arange(32) * 8] = level
    check(g, row, 8)
    row = torch.full((vocab,), level - 20.0)
    row[0] = level
    check(g, row, 0)
