"""The losses against their definition in 64 bits on the device: what the GPU tests of larger sizes share.

Bounds are those of test_gpu_losses.py. With c the row's shift, a term that counts has |x k - c| <= 64 in these
tests, so that it carries at most 68 * 2^-23 relative and its sum less than 4e-5; the rounded k moves all of a row's
logits by the same factor, at most 2^-24 of their difference. A slope of a preference loss moves with its log ratio:
beta times at most 320 rows' 4e-5, below 1.3e-3 of itself at beta = 0.1.
"""

import torch

LP_ABS, LP_REL, GRAD = 4e-5, 2.0 ** -23, 2e-4


def log_probs(x, labels, tau):
    """lp and the softmax of every row in 64 bits (0 and zeros where a label is negative)."""
    z = x.double() / tau
    z = z - z.amax(1, keepdim=True)
    z = z - z.exp().sum(1, keepdim=True).log()
    lp = z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    return torch.where(labels >= 0, lp, 0.0), z.exp_()


def check_logp(got, want):
    err = (got.double() - want).abs()
    assert (err <= LP_ABS + LP_REL * want.abs()).all(), float((err - LP_REL * want.abs()).max())


def check_gradient(got, up, p, labels, tau, rel=GRAD):
    """`got` against up * (onehot - p) / tau, up: dL/dlp."""
    rows = torch.arange(len(labels), device="cuda")
    own = torch.where(labels >= 0, 1.0, 0.0).double()
    at = labels.clamp(min=0)
    want = p * (-up * own / tau)[:, None]
    want[rows, at] += up * own / tau
    bound = p * (rel * up.abs() / tau)[:, None]
    bound[rows, at] += rel * up.abs() / tau
    if got.dtype == torch.bfloat16:
        bound += 2.0 ** -8 * want.abs()
    over = (got.double() - want).abs() - bound - 1e-37
    assert (over <= 0).all(), float(over.max())


def check_all(g, x, labels, tau):
    """The three losses on these rows: four sequences, ratios of 1.1, log ratios of the pairs near 0."""
    rows = len(labels)
    start = torch.tensor([0, rows // 4, rows // 2, 3 * rows // 4, rows], device="cuda")
    lp, p = log_probs(x, labels, tau)
    has = (labels >= 0).double()
    check_logp(g.ar_token_logp(x, labels, temperature=tau), lp)

    old = (lp - 0.09531018).float()
    adv = torch.where(torch.arange(rows, device="cuda") % 3 == 0, -1.0, 1.0)
    r = torch.exp(lp - old.double())
    stats, got, d = g.ar_policy_loss(x, labels, old, adv, start, clip_low=0.2, clip_high=0.2, temperature=tau)
    check_logp(got, lp)
    up = -r * adv.double() * has / has.sum()
    check_gradient(d, up, p, labels, tau)
    assert abs(float(stats[0]) - float(up.sum())) <= 1e-4 * float(up.abs().sum())
    own = x.clone()
    again = g.ar_policy_loss(own, labels, old, adv, start, clip_low=0.2, clip_high=0.2, temperature=tau, dlogits=own)[2]
    # (a row's alignment decides the order of its sum: same stride, same bits)
    if own.stride() == x.stride() and (own.data_ptr() - x.data_ptr()) % 16 == 0:
        assert torch.equal(again, d)
    else:
        check_gradient(again, up, p, labels, tau)

    noise = torch.randn(rows, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 0.1
    ref = (lp + noise).float()
    stats, ratios, got, d = g.ar_preference_loss(x, labels, ref, start, beta=0.1, temperature=tau)
    check_logp(got, lp)
    gap = (lp - ref.double()) * has
    want = torch.stack([gap[int(a):int(b)].sum() for a, b in zip(start[:-1], start[1:])])
    n = torch.stack([has[int(a):int(b)].sum() for a, b in zip(start[:-1], start[1:])])
    assert ((ratios.double() - want).abs() <= n * (LP_ABS + LP_REL * lp.abs().max()) + 1e-6 * want.abs()).all()
    z = 0.1 * (want[0::2] - want[1::2])
    slope = torch.stack([-torch.sigmoid(-z), torch.sigmoid(-z)], 1).reshape(-1) * 0.1 / 2
    up = torch.repeat_interleave(slope, start[1:] - start[:-1]) * has
    check_gradient(d, up, p, labels, tau, rel=1.5e-3)
    assert g.ar_device_status() == g.AR_OK
