"""The losses where a row is the work of several CTAs that hold it in registers, or read it twice, on a GB300."""

import math

import pytest
import torch

from _loss_checks import check_all, check_logp, log_probs

pytestmark = pytest.mark.gpu

# (rows, vocab, type): clusters of 2, 4, 8 and 8 CTAs; rows beyond what eight CTAs hold, few of them and (the policy
# loss alone: the others stream) many
ROWS = [(100, 32000, torch.bfloat16), (60, 32000, torch.bfloat16), (20, 32000, torch.float32),
        (16, 131072, torch.float32), (5, 262147, torch.float32), (40, 300001, torch.bfloat16),
        (620, 140003, torch.float32)]


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def inputs(rows, vocab, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).to(dtype)
    labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    labels[::5] = -100
    return x, labels


@pytest.mark.parametrize("rows,vocab,dtype", ROWS)
def test_rows_of_several_ctas(g, rows, vocab, dtype):
    x, labels = inputs(rows, vocab, dtype, seed=vocab)
    check_all(g, x, labels, 0.8)
    first = g.ar_token_logp(x, labels)
    lp = first - 0.1
    start = torch.tensor([0, rows // 2, rows], device="cuda")
    pref = g.ar_preference_loss(x, labels, lp, start)
    pol = g.ar_policy_loss(x, labels, lp, lp, start)
    for _ in range(10):
        assert torch.equal(first, g.ar_token_logp(x, labels))
        assert all(torch.equal(a, b) for a, b in zip(pol, g.ar_policy_loss(x, labels, lp, lp, start)))
        assert all(torch.equal(a, b) for a, b in zip(pref, g.ar_preference_loss(x, labels, lp, start)))


@pytest.mark.parametrize("rows,vocab,dtype", ROWS[:5])
def test_sums_taken_twice(g, rows, vocab, dtype):
    """Rows at the type's lowest or highest value, where x / tau is not finite and the sum is taken again."""
    x, labels = inputs(rows, vocab, dtype, seed=1)
    labels[:4] = 3
    x[0] = torch.finfo(dtype).min
    x[1] = torch.finfo(dtype).max
    x[2] = torch.finfo(dtype).min
    x[2, vocab // 2:] = -float("inf")
    x[3, 3] = torch.finfo(dtype).max
    x[3, vocab - 1] = torch.finfo(dtype).max
    lp = g.ar_token_logp(x, labels, temperature=0.5)
    want = [-math.log(vocab), -math.log(vocab), -math.log(vocab // 2), -math.log(2)]
    assert (lp[:4].double().cpu() - torch.tensor(want, dtype=torch.float64)).abs().max() < 4e-5
    check_logp(lp[4:], log_probs(x[4:], labels[4:], 0.5)[0])
    up = -1.0 / rows
    every = torch.where(labels < 0, 0, labels)
    every[:4] = 3
    old = g.ar_token_logp(x, every, temperature=0.5)
    _, got, d = g.ar_policy_loss(x, every, old, torch.ones(rows, device="cuda"), temperature=0.5)
    assert torch.equal(got, old)
    for row, n in ((0, vocab), (1, vocab), (2, vocab // 2)):
        p = torch.zeros(vocab, dtype=torch.float64, device="cuda")
        p[:n] = 1 / n
        want = -p * up / 0.5
        want[3] += up / 0.5
        assert ((d[row].double() - want).abs() <= (2.0 ** -8 if dtype == torch.bfloat16 else 2e-4) * want.abs()).all()
