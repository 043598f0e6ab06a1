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


def farthest(kind, lo, hi):
    """Scores between lo and hi whose product with log2 e is the farthest from an fp32 number."""
    x = torch.linspace(lo, hi, 4001).to(kind).double().numpy()
    k = float(np.float32(np.log2(np.e)))
    off = np.abs(x * k - (x * k).astype(np.float32))
    return float(x[np.argmax(off)])


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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [8192, 32003, 131072])
@pytest.mark.parametrize("low,high,room", [(0.0, (45.0, 60.0), FAR), (-30.0, (15.0, 35.0), FAR), (0.0, (80.0, 88.0), FAR),
                                           (0.0, (14.0, 18.0), NEAR), (-10.0, (4.0, 11.0), NEAR)])
def test_one_token_far_above_the_rest(g, dtype, vocab, low, high, room):
    """Behind groups of scores far below, one token that has all the weight: its log-probability is 0 but for theirs."""
    x = farthest(KINDS[dtype], *high)
    for token in (2048 + 77, vocab // 2 - 3, vocab - 1):
        row = torch.full((vocab,), low, dtype=KINDS[dtype])
        row[token] = x
        check(g, row, token, room)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [8192, 32003])
@pytest.mark.parametrize("mask", ["-inf", "lowest"])
@pytest.mark.parametrize("level", [-68.0, -30.0, 60.0])
def test_masked_groups_before_scores_far_from_zero(g, dtype, vocab, mask, level):
    """Stretches of a row are ruled out; in the others one token, and all others 20 to 21 below it: shares of 1e-9 each, and
    together one of 5e-6 or more."""
    kind = KINDS[dtype]
    rng = np.random.default_rng(vocab)
    for stretch in (8, 2048, vocab // 2):
        row = torch.from_numpy(level - rng.uniform(20.0, 21.0, vocab)).to(kind)
        masked = (torch.arange(vocab) // stretch) % 2 == 0
        row[masked] = -float("inf") if mask == "-inf" else torch.finfo(kind).min
        free = torch.nonzero(~masked)[:, 0]
        for token in free[:: len(free) // 5].tolist():
            one = row.clone()
            one[token] = level
            check(g, one, token)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_low_scores_behind_masked_ones(g, dtype):
    """Every other stretch of 2048 is ruled out. In the rest 8192 tokens, one a thread of the sums, and eight million
    others with a share of 1e-8 of theirs: together 1e-5."""
    vocab = 1 << 24
    row = torch.full((vocab,), -87.5, dtype=KINDS[dtype])
    at = torch.arange(vocab)
    row[(at % (1 << 19) // 2048 == 1) & (at % 8 == 0)] = -69.0
    row[at // 2048 % 2 == 0] = -float("inf")
    check(g, row, 2048 + 8 * 77)


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
