"""The losses where they stream rows (more than 32 KB a row, more than 512 rows and at least four rows times CTAs for
each SM), on a GB300, against their definition in 64 bits on the device."""

import math

import pytest
import torch

from _loss_checks import check_all, check_gradient, check_logp, log_probs

pytestmark = pytest.mark.gpu

# (rows, vocab, type): the policy loss in clusters of 1, 1, 2, 4 and 8 CTAs a row
STREAMED = [(640, 16500, torch.bfloat16), (640, 8300, torch.float32), (640, 40003, torch.bfloat16),
            (620, 100003, torch.bfloat16), (620, 100003, torch.float32)]


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def normal(rows, vocab, dtype, shift=0, pad=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, shift + vocab + pad, generator=gen, device="cuda") * 3).to(dtype)[:, shift:shift + vocab]
    labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    edges = torch.arange(0, rows, 9, device="cuda")  # first and last elements, outside the vectors or not
    labels[edges] = torch.where(edges % 2 == 0, edges // 9 % 8, vocab - 1 - edges // 9 % 8)
    labels[::4] = -100
    return x, labels


@pytest.mark.parametrize("shift,pad", [(0, 0), (3, 2)])
@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_streamed_rows(g, rows, vocab, dtype, shift, pad):
    x, labels = normal(rows, vocab, dtype, shift, pad, seed=vocab + shift)
    check_all(g, x, labels, 0.9)


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_gradient_over_the_logits(g, rows, vocab, dtype):
    """In place and apart, the same bits, call after call."""
    x, labels = normal(rows, vocab, dtype, seed=2)
    start = torch.tensor([0, 99, 300, 301, rows], device="cuda")
    lp = g.ar_token_logp(x, labels)
    for loss, args in ((g.ar_policy_loss, (lp - 0.1, lp, start)), (g.ar_preference_loss, (lp + 0.1, start))):
        want = loss(x, labels, *args)
        for _ in range(4):
            own = x.clone()
            got = loss(own, labels, *args, dlogits=own)
            assert got[-1].data_ptr() == own.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.ar_device_status() == g.AR_OK


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_extreme_values(g, rows, vocab, dtype):
    """Rows whose sums are taken again, in every CTA of a cluster, among others whose are not."""
    low, top = torch.finfo(dtype).min, torch.finfo(dtype).max
    x, labels = normal(rows, vocab, dtype, seed=3)
    labels[:9] = 5
    x[0] = low                           # uniform
    x[1, 9:] = low                       # uniform over nine
    x[1, :9] = 0.0
    x[2] = -float("inf")                 # no distribution
    x[3, vocab - 1] = float("nan")
    x[4, 0] = float("inf")
    labels[5] = vocab + 3
    x[6] = top                           # uniform
    x[7] = low
    x[7, 5] = x[7, vocab - 7] = top      # uniform over two, far apart
    x[8] = -300.0                        # below what a thread's shift takes in at first
    x[8, 5] = -298.0
    want = [-math.log(vocab), -math.log(9), *[math.nan] * 4, -math.log(vocab), -math.log(2),
            2 - math.log(vocab - 1 + math.exp(2.0))]
    lp = g.ar_token_logp(x, labels)
    for i, v in enumerate(want):
        assert math.isnan(lp[i]) if math.isnan(v) else abs(float(lp[i]) - v) < 4e-5, (i, lp[i], v)
    check_logp(lp[9:], log_probs(x[9:], labels[9:], 1.0)[0])
    start = torch.tensor([0, rows], device="cuda")
    _, got, d = g.ar_policy_loss(x, labels, torch.nan_to_num(lp, 0.0), torch.ones(rows, device="cuda"), start)
    check_logp(torch.nan_to_num(got), torch.nan_to_num(lp).double())
    assert torch.isnan(d[2:6]).all() and torch.isfinite(d[6:]).all() and torch.isfinite(d[:2]).all()
    even = torch.full((1, vocab), 1 / vocab, dtype=torch.float64, device="cuda")
    up = torch.full((1,), -1.0 / int((labels >= 0).sum()), dtype=torch.float64, device="cuda")
    for i in (0, 6):
        check_gradient(d[i:i + 1], up, even, labels[i:i + 1], 1.0)


# logit / temperature of the two entries that are left in a row; the first is among the first
# vectors of its thread, the second is not, and its thread's first vectors hold the mask
PAIRS = [(43.75, 43.75), (43.5, 44.0), (44.0, 46.0), (44.0, 50.0), (50.0, 44.0), (60.0, 61.0), (120.0, 119.0),
         (-150.0, -151.0), (3.0, 2.0), (-30.0, 43.0)]


@pytest.mark.parametrize("low", ["inf", "lowest", "far"])
@pytest.mark.parametrize("tau", [1.0, 0.25])
@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_masked_rows_of_large_logits(g, rows, vocab, dtype, tau, low):
    """Nothing is lost where a mask hides a thread's first vectors and the logits that are left are large."""
    fill = {"inf": -float("inf"), "lowest": torch.finfo(dtype).min, "far": -400.0 * tau}[low]
    x = torch.full((rows, vocab), fill, dtype=dtype, device="cuda")
    width = 1024 * (8 if dtype == torch.bfloat16 else 4)  # two vectors a thread
    t = torch.arange(rows, device="cuda")
    pairs = torch.tensor(PAIRS, device="cuda")[t % len(PAIRS)] * tau
    first, late = 5 + t * 7 % (width - 50), width + 10 + t * 13 % (min(width, vocab - width) - 50)
    x[t, first] = pairs[:, 0].to(dtype)
    x[t, late] = pairs[:, 1].to(dtype)
    labels = torch.where(t % 2 == 0, first, late)
    labels[::9] = -100
    check_all(g, x, labels, tau)


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_masked_start_of_the_rows(g, rows, vocab, dtype):
    """All of the first vectors but one entry ruled out, the rest ten nats below it."""
    width = 1024 * (8 if dtype == torch.bfloat16 else 4)
    x = torch.full((rows, vocab), 33.25, dtype=dtype, device="cuda")
    x[:, :width] = -float("inf")
    t = torch.arange(rows, device="cuda")
    x[t, 3 + t] = 43.5
    labels = torch.where(t % 2 == 0, 3 + t, width + 20 + t)
    labels[::5] = -1
    check_all(g, x, labels, 1.0)


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_forced_tokens(g, rows, vocab, dtype):
    """A token at the type's highest value has all of its row's probability, wherever in the row it is."""
    x, labels = normal(rows, vocab, dtype, seed=6)
    t = torch.arange(rows, device="cuda")
    labels = t * 131 % vocab
    x[t, labels] = torch.finfo(dtype).max
    assert not g.ar_token_logp(x, labels).any()
    old = torch.zeros(rows, device="cuda")
    stats, lp, d = g.ar_policy_loss(x, labels, old, old + 1)
    assert not lp.any() and not d.any() and abs(float(stats[0]) + 1) < 1e-6


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_rows_outside_the_sequences(g, rows, vocab, dtype):
    """Labelled rows of no sequence have no gradient, whatever they hold."""
    x, labels = normal(rows, vocab, dtype, seed=4)
    x[:, 3::7] = -float("inf")
    x[1], x[2, 7], x[3] = float("nan"), float("inf"), -float("inf")
    x[rows - 2, vocab - 1], x[rows - 1] = float("nan"), torch.finfo(dtype).min
    start = torch.tensor([5, 300, 300, 400, rows - 10], device="cuda")
    labels[:5] = labels[rows - 10:] = 4
    labels = torch.where(labels % 7 == 3, labels + 1, labels)  # none ruled out
    labels[labels >= vocab] = 0
    lp = g.ar_token_logp(x, labels)
    check_logp(lp[5:rows - 2], log_probs(x[5:rows - 2], labels[5:rows - 2], 1.0)[0])
    assert torch.isnan(lp[1:4]).all() and torch.isnan(lp[rows - 2])
    other = torch.nan_to_num(lp, 0.0)
    calls = [lambda y, **kw: g.ar_policy_loss(y, labels, other - 0.1, other + 5, start, reduction=r, **kw)
             for r in ("token", "sequence")] + [lambda y, **kw: g.ar_preference_loss(y, labels, other + 0.1, start, **kw)]
    for call in calls:
        *stats, _, d = call(x)
        assert torch.isfinite(stats[0]).all() and torch.isfinite(d).all()
        assert not d[:5].any() and not d[rows - 10:].any() and d[5:rows - 10].any()
        own = x.clone()
        assert torch.equal(call(own, dlogits=own)[-1], d)


@pytest.mark.parametrize("tau", [0.1, 0.01])
@pytest.mark.parametrize("fill", [None, -1e4, -float("inf")])
@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_low_temperatures(g, rows, vocab, dtype, fill, tau):
    """Logits hundreds apart over the temperature, and the same behind a mask that hides a thread's first vectors."""
    x, labels = normal(rows, vocab, dtype, seed=7)
    if fill is not None:
        x[:, :1024 * (8 if dtype == torch.bfloat16 else 4)] = fill
    best = x.topk(2, 1).indices  # (a log-probability of hundreds would bring in its own rounding)
    labels = torch.where(labels < 0, labels, best[torch.arange(rows, device="cuda"), labels % 2])
    check_all(g, x, labels, tau)
