"""The losses on a GB300 against their oracle in 64 bits.

Bounds, from the kernels' arithmetic. With R = max_j |x_j - max x| log2(e) / tau
(at most 130 in these tests): every term 2^(x k - c) carries at most
(R + 4) * 2^-23 relative (one FMA rounding and the rounded k in the exponent,
two ulp of the exponential), its fp32 sum at most (vocab / 512 + 24) * 2^-24
more: below 4e-5 in all for the sizes here. So
  |lp - exact|   <= 4e-5 + 2^-23 |lp|
and the slope dL/dlp moves by at most that much times (r |A| + beta e^b + its
own value), the softmax by 4e-5 of itself twice: 2e-4 of the sum of the
magnitudes that make up each gradient element. bf16 gradients add half an ulp.
"""

import numpy as np
import pytest
import torch

from oracle import losses

pytestmark = pytest.mark.gpu

LP_ABS, LP_REL, GRAD = 4e-5, 2.0 ** -23, 2e-4
CLIP = (0.2, 0.3)


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def make(rows, vocab, dtype, seed=0, shift=0, pad=0, masked=0.25, ruled=0.0, n_seq=1, spread=3.0):
    """Inputs on the device: logits as a view `shift` columns into rows of vocab + shift + pad."""
    rng = np.random.default_rng(seed)
    t = torch.tensor(rng.normal(size=(rows, shift + vocab + pad)) * spread, dtype=dtype, device="cuda")
    x = t[:, shift:shift + vocab]
    labels = rng.integers(0, vocab, rows)
    if ruled:
        out = torch.tensor(rng.random((rows, vocab)) < ruled, device="cuda")
        out[torch.arange(rows), torch.tensor(labels, device="cuda")] = False
        x.masked_fill_(out, -np.inf)
    labels[rng.random(rows) < masked] = -100
    cuts = np.sort(rng.integers(0, rows + 1, n_seq - 1))
    start = np.concatenate([[0], cuts, [rows]]).astype(np.int64)
    host = x.double().cpu().numpy()
    now = losses.token_logp(host, labels)
    ratio = np.array([0.5, 0.7, 0.9, 1.0, 1.1, 1.25, 1.4, 2.0])[rng.integers(0, 8, rows)]
    old = (now - np.log(ratio)).astype(np.float32)
    ref = (now + rng.normal(size=rows) * 0.5).astype(np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    dev = {k: torch.tensor(v, device="cuda") for k, v in dict(labels=labels, old=old, ref=ref, adv=adv,
                                                                 start=start).items()}
    return x, host, dev, dict(labels=labels, old=old, ref=ref, adv=adv, start=start)


def check_logp(got, want):
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (err <= LP_ABS + LP_REL * np.abs(want)).all(), err.max()


def check_gradient(got, want, host, labels, parts, temperature=1.0):
    """parts[t]: the sum of the magnitudes that make up dL/dlp of row t."""
    p = np.zeros(host.shape)
    rows = np.nonzero(labels >= 0)[0]
    p[rows] = np.exp(losses.log_softmax(host[rows], temperature))
    p[rows, labels[rows]] += 1.0
    bound = GRAD / temperature * parts[:, None] * p + 1e-37
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()


def policy(g, x, host, dev, cpu, kl=0.1, mean="token", temperature=1.0, **kw):
    stats, logp, d = g.ar_policy_loss(
        x, dev["labels"], dev["old"], dev["adv"], dev["start"], ref_logp=dev["ref"] if kl else None, clip_low=CLIP[0],
        clip_high=CLIP[1], kl_coef=kl, reduction=mean, temperature=temperature, **kw)
    want = losses.policy_loss(host, cpu["labels"], cpu["old"], cpu["adv"], cpu["start"],
                              ref=cpu["ref"] if kl else None, clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=kl,
                              mean=mean, temperature=temperature, denominator=kw.get("denominator", 0.0),
                              grad_scale=kw.get("grad_scale", 1.0))
    check_logp(logp, want["logp"])
    r = np.exp(want["logp"] - cpu["old"])
    b = np.exp(cpu["ref"] - want["logp"]) if kl else 0 * r
    parts = np.abs(want["weights"]) * (r * np.abs(cpu["adv"]) + kl * (1 + b)) * abs(kw.get("grad_scale", 1.0))
    if d is not None:
        check_gradient(d, want["dlogits"], host, cpu["labels"], parts, temperature)
    size = np.array([(want["weights"] * (r * np.abs(cpu["adv"]) + kl * (1 + b))).sum(),
                     (want["weights"] * r * np.abs(cpu["adv"])).sum(), (want["weights"] * (1 + b)).sum(), 1.0])
    assert (np.abs(stats.double().cpu().numpy() - want["stats"]) <= 1e-4 * size + 1e-12).all(), (stats, want["stats"])
    return stats, logp, d


SIZES = [(1, 1), (5, 2), (3, 7), (64, 8), (7, 33), (40, 1000), (9, 4099), (6, 32000), (3, 50021), (2, 131072)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_policy(g, rows, vocab, dtype):
    policy(g, *make(rows, vocab, dtype, seed=vocab, n_seq=3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 2), (4, 4), (0, 7), (7, 1)])
def test_policy_strides_and_alignment(g, shift, pad, dtype):
    inputs = make(23, 2011, dtype, seed=shift, shift=shift, pad=pad, n_seq=4)
    a = policy(g, *inputs, mean="sequence", temperature=0.7)[2]
    # the gradient may have another stride and alignment than the logits
    room = torch.full((23, 2011 + 5), 7.0, dtype=dtype, device="cuda")
    b = policy(g, *inputs, mean="sequence", temperature=0.7, dlogits=room[:, 3:2014])[2]
    assert torch.equal(a, b)
    assert (room[:, :3] == 7).all() and (room[:, 2014:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [5, 2011, 32000])
def test_policy_in_place(g, vocab, dtype):
    x, host, dev, cpu = make(17, vocab, dtype, seed=5, n_seq=2)
    apart = policy(g, x, host, dev, cpu)[2]
    own = x.clone()
    d = policy(g, own, host, dev, cpu, dlogits=own)[2]
    assert d.data_ptr() == own.data_ptr() and torch.equal(d, apart)


def test_policy_options(g):
    inputs = make(50, 777, torch.float32, seed=9, n_seq=5)
    policy(g, *inputs, kl=0.0)
    policy(g, *inputs, denominator=123.0, grad_scale=-2.5)
    policy(g, *inputs, mean="sequence", denominator=7.0)
    assert policy(g, *inputs, grad=False)[2] is None


@pytest.mark.parametrize("mean", ["token", "sequence"])
def test_masks_that_leave_nothing(g, mean):
    x, host, dev, cpu = make(12, 100, torch.float32, masked=1.0, n_seq=3)
    stats, logp, d = policy(g, x, host, dev, cpu, mean=mean)
    assert not stats.any() and not logp.any() and not d.any()
    # no rows at all
    none = x[:0]
    empty = {k: v[:0] for k, v in dev.items()}
    stats, logp, d = g.ar_policy_loss(none, empty["labels"], empty["old"], empty["adv"],
                                      torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert not stats.any() and logp.shape == (0,) and d.shape == (0, 100)
    assert g.ar_token_logp(none, empty["labels"]).shape == (0,)


def test_masked_rows_are_not_read(g):
    x, host, dev, cpu = make(16, 300, torch.float32, seed=2, n_seq=2)
    clean = policy(g, x, host, dev, cpu)
    off = dev["labels"] < 0
    x[off] = float("nan")
    for k in ("old", "ref", "adv"):
        dev[k][off] = float("nan")
    stats, logp, d = g.ar_policy_loss(x, dev["labels"], dev["old"], dev["adv"], dev["start"], ref_logp=dev["ref"],
                                      clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=0.1)
    assert torch.equal(stats, clean[0]) and torch.equal(logp, clean[1]) and torch.equal(d, clean[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ruled", [0.5, 1.0])
def test_ruled_out_tokens(g, dtype, ruled):
    """Entries of -inf have probability 0; with all others ruled out the label has probability 1."""
    x, host, dev, cpu = make(8, 1500, dtype, ruled=ruled, n_seq=2)
    _, logp, d = policy(g, x, host, dev, cpu)
    assert not d[torch.isinf(x)].any()
    if ruled == 1.0:
        assert (logp.abs() < 1e-6).all()


def test_lowest_values_infinities_and_nan(g):
    x = torch.zeros(6, 70, device="cuda")
    x[0, 1:] = torch.finfo(torch.float32).min  # a mask of the type's lowest value: probability 0
    x[1] = torch.finfo(torch.float32).min      # every entry the lowest: uniform
    x[2] = -float("inf")                       # no distribution
    x[3, 5] = float("inf")
    x[4, 69] = float("nan")
    labels = torch.zeros(6, dtype=torch.int64, device="cuda")
    labels[5] = 70                             # outside the vocabulary
    lp = g.ar_token_logp(x, labels).cpu().numpy()
    assert lp[0] == 0.0 and abs(lp[1] + np.log(70)) < 1e-6 and np.isnan(lp[2:]).all()
    x[1, 40:] = -float("inf")
    x[0, 1:] = torch.finfo(torch.float32).max
    lp = g.ar_token_logp(x, labels).cpu().numpy()
    assert lp[0] == -np.inf or lp[0] < -1e38  # the others are the highest value
    assert abs(lp[1] + np.log(40)) < 1e-6
    # the gradient of such rows: softmax 1/40 on the lowest values, and what the two passes of a pair agree on
    ref = torch.zeros(6, device="cuda")
    start = torch.tensor([0, 1, 2], device="cuda")
    x[0] = 0.0
    d = g.ar_preference_loss(x[:2], labels[:2], ref[:2], start, beta=1.0)[3]
    c = float(d[1, 0]) / (1 - 1 / 40)
    assert abs(c) > 0.1 and torch.allclose(d[1, 1:40], torch.full((39,), -c / 40, device="cuda"), rtol=1e-5)
    assert not d[1, 40:].any()


def test_sequences_that_do_not_cover_the_rows(g):
    x, host, dev, cpu = make(20, 60, torch.float32, masked=0.1)
    start = np.array([3, 3, 9, 15], np.int64)
    cpu["start"], dev["start"] = start, torch.tensor(start, device="cuda")
    _, logp, d = policy(g, x, host, dev, cpu, mean="sequence")
    assert not d[:3].any() and not d[15:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_token_logp(g, rows, vocab, dtype):
    x, host, dev, cpu = make(rows, vocab, dtype, seed=rows, ruled=0.1)
    check_logp(g.ar_token_logp(x, dev["labels"], temperature=0.6), losses.token_logp(host, cpu["labels"], 0.6))


def preference(g, x, host, dev, cpu, temperature=1.0, **kw):
    stats, ratios, logp, d = g.ar_preference_loss(x, dev["labels"], dev["ref"], dev["start"], temperature=temperature,
                                                  **kw)
    names = dict(loss="form")
    okw = {names.get(k, k): v for k, v in kw.items() if k not in ("grad", "dlogits")}
    want = losses.preference_loss(host, cpu["labels"], cpu["ref"], cpu["start"], temperature=temperature, **okw)
    check_logp(logp, want["logp"])
    labelled = np.array([(cpu["labels"][a:b] >= 0).sum() for a, b in zip(cpu["start"][:-1], cpu["start"][1:])])
    over = np.maximum(labelled, 1) if kw.get("length_normalized") else 1
    lp_err = (LP_ABS + LP_REL * np.abs(want["logp"]).max(initial=0)) * labelled / over
    assert (np.abs(ratios.double().cpu().numpy() - want["ratios"]) <= lp_err + 1e-6 * np.abs(want["ratios"])).all()
    beta = kw.get("beta", 0.1)
    z_err = beta * (lp_err[0::2] + lp_err[1::2]).max(initial=0)  # dL/dz moves by at most 2 per unit of z
    assert (np.abs(stats.double().cpu().numpy() - want["stats"])[:3]
            <= z_err * np.array([3 * (1 + np.abs(want["ratios"]).max(initial=0) * beta), 1, 1])
            + 1e-5 * np.abs(want["stats"][:3]) + 1e-7).all(), (stats, want["stats"])
    assert abs(float(stats[3]) - want["stats"][3]) < 1e-6
    if d is not None:
        seq = np.searchsorted(cpu["start"][1:], np.arange(len(cpu["labels"])), side="right")
        pairs = kw.get("denominator", 0.0) or len(labelled) // 2
        per_row = beta / pairs / (over[np.minimum(seq, len(labelled) - 1)] if np.ndim(over) else 1)
        parts = np.abs(want["slope"]) + 2 * z_err / GRAD * per_row * abs(kw.get("grad_scale", 1.0))
        check_gradient(d, want["dlogits"], host, cpu["labels"], parts, temperature)
    return stats, ratios, logp, d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_preference(g, rows, vocab, dtype):
    preference(g, *make(rows, vocab, dtype, seed=rows + vocab, n_seq=4))


@pytest.mark.parametrize("kw", [dict(loss="sigmoid", label_smoothing=0.1), dict(loss="square", target=0.7),
                                dict(loss="square", length_normalized=True), dict(length_normalized=True, beta=2.0),
                                dict(denominator=64.0, grad_scale=0.5)])
@pytest.mark.parametrize("shift", [0, 3])
def test_preference_options(g, kw, shift):
    preference(g, *make(61, 501, torch.float32, seed=4, n_seq=6, shift=shift, pad=2), temperature=1.3, **kw)


def test_preference_in_place_and_forward_only(g):
    x, host, dev, cpu = make(30, 2011, torch.bfloat16, seed=8, n_seq=4)
    apart = preference(g, x, host, dev, cpu)
    assert preference(g, x, host, dev, cpu, grad=False)[3] is None
    own = x.clone()
    d = preference(g, own, host, dev, cpu, dlogits=own)[3]
    assert torch.equal(d, apart[3])


# Calls with many long rows, which are streamed: (rows, vocab, dtype); the policy loss in clusters of 1, 1, 4 and
# 2 CTAs a row.
STREAMED = [(650, 8200, torch.bfloat16), (700, 5001, torch.float32), (160, 50021, torch.float32),
            (330, 40003, torch.bfloat16), (640, 16500, torch.bfloat16), (650, 8300, torch.float32)]


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
@pytest.mark.parametrize("shift", [0, 3])
def test_streamed_rows(g, rows, vocab, dtype, shift):
    inputs = make(rows, vocab, dtype, seed=rows, shift=shift, pad=2, n_seq=6, ruled=0.02)
    x, host, dev, cpu = inputs
    check_logp(g.ar_token_logp(x, dev["labels"], temperature=0.9), losses.token_logp(host, cpu["labels"], 0.9))
    stats, logp, d = policy(g, *inputs, mean="sequence", temperature=0.9)
    preference(g, *inputs, temperature=1.1, length_normalized=True)
    # gradients over the logits, and at another alignment
    room = torch.full((rows, vocab + 5), 7.0, dtype=dtype, device="cuda")
    assert torch.equal(d, policy(g, *inputs, mean="sequence", temperature=0.9, dlogits=room[:, 4:vocab + 4])[2])
    assert (room[:, :4] == 7).all() and (room[:, vocab + 4:] == 7).all()
    # (at the logits' own alignment: sums run in an order that depends on it)
    own = torch.empty(rows, shift + vocab + 2, dtype=dtype, device="cuda")[:, shift:shift + vocab]
    own.copy_(x)
    pref = preference(g, *inputs, beta=0.3)[3]
    got = g.ar_preference_loss(own, dev["labels"], dev["ref"], dev["start"], beta=0.3, dlogits=own)[3]
    assert torch.equal(got, pref)
    own.copy_(x)
    again = g.ar_policy_loss(own, dev["labels"], dev["old"], dev["adv"], dev["start"], ref_logp=dev["ref"],
                             clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=0.1, reduction="sequence", temperature=0.9,
                             dlogits=own)
    assert torch.equal(again[2], d) and torch.equal(again[0], stats) and torch.equal(again[1], logp)
    assert g.ar_device_status() == g.AR_OK


@pytest.mark.parametrize("rows,vocab,dtype", STREAMED)
def test_streamed_rows_of_extreme_values(g, rows, vocab, dtype):
    low = torch.finfo(dtype).min
    x, host, dev, cpu = make(rows, vocab, dtype, seed=1, n_seq=2, masked=0.0)
    dev["labels"][:6] = 5
    x[0] = low               # uniform
    x[1, 9:] = low           # uniform over nine
    x[1, :9] = 0.0
    x[2] = -float("inf")
    x[3, vocab - 1] = float("nan")
    x[4, 0] = float("inf")
    dev["labels"][5] = vocab + 3
    lp = g.ar_token_logp(x, dev["labels"]).cpu().numpy()
    assert abs(lp[0] + np.log(vocab)) < 1e-5 and abs(lp[1] + np.log(9)) < 1e-6 and np.isnan(lp[2:6]).all()
    check_logp(torch.tensor(lp[6:]), losses.token_logp(host[6:], cpu["labels"][6:]))
    d = g.ar_policy_loss(x, dev["labels"], dev["old"], dev["adv"], dev["start"])[2].float()
    assert torch.isnan(d[2:6]).all() and torch.isfinite(d[6:]).all()
    # rows that a mask takes out are not read
    dev["labels"][:6] = -1
    stats, _, d = g.ar_policy_loss(x, dev["labels"], dev["old"], dev["adv"], dev["start"])
    assert not d[:6].any() and torch.isfinite(stats).all()


def test_streamed_rows_longer_than_the_ring(g):
    """Rows of 200 and 400 KB; the definition in 64 bits on the device. Bounds as at the top."""
    for vocab, dtype in ((100003, torch.bfloat16), (100003, torch.float32)):
        rows = 620
        gen = torch.Generator(device="cuda").manual_seed(vocab)
        x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).to(dtype)
        labels = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        labels[::7] = -1
        start = torch.tensor([0, 100, 333, 400, rows], device="cuda")
        ref = torch.full((rows,), -9.0, device="cuda")
        logp = torch.log_softmax(x.double(), 1).gather(1, labels.clamp(min=0)[:, None])[:, 0]
        logp = torch.where(labels >= 0, logp, 0.0)
        check_logp(g.ar_token_logp(x, labels), logp.cpu().numpy())
        stats, ratios, got, d = g.ar_preference_loss(x, labels, ref, start, beta=0.01)
        check_logp(got, logp.cpu().numpy())
        gap = torch.where(labels >= 0, logp + 9.0, 0.0)
        want = torch.stack([gap[a:b].sum() for a, b in zip([0, 100, 333, 400], [100, 333, 400, rows])])
        z = 0.01 * (want[0::2] - want[1::2])
        slope = torch.stack([-torch.sigmoid(-z), torch.sigmoid(-z)], 1).reshape(-1) * 0.01 / 2
        up = torch.repeat_interleave(slope, torch.tensor([100, 233, 67, rows - 400], device="cuda"))
        up = torch.where(labels >= 0, up, 0.0)
        exact = torch.softmax(x.double(), 1) * -up[:, None]
        exact[torch.arange(rows), labels.clamp(min=0)] += up
        # the slope moves by at most beta * 620 * 1e-4 of itself
        bound = 1e-3 * exact.abs() + (2.0 ** -8 if dtype == torch.bfloat16 else 0) * exact.abs() + 1e-3 * up.abs()[:, None] * GRAD
        assert ((d.double() - exact).abs() <= bound + 1e-12).all()
        old, adv = logp.float() - 0.05, torch.ones(rows, device="cuda")
        _, got, d = g.ar_policy_loss(x, labels, old, adv)
        check_logp(got, logp.cpu().numpy())
        up = torch.where(labels >= 0, -torch.exp(logp - old.double()) / (labels >= 0).sum(), 0.0)
        exact = torch.softmax(x.double(), 1) * -up[:, None]
        exact[torch.arange(rows), labels.clamp(min=0)] += up
        bound = 1e-3 * exact.abs() + (2.0 ** -8 if dtype == torch.bfloat16 else 0) * exact.abs() + up.abs()[:, None] * GRAD
        assert ((d.double() - exact).abs() <= bound + 1e-12).all()
        assert g.ar_device_status() == g.AR_OK


def test_streamed_rows_outside_the_sequences(g):
    rows, vocab = 700, 8200
    x, host, dev, cpu = make(rows, vocab, torch.bfloat16, seed=3, masked=0.1)
    start = np.array([5, 300, 300, 690], np.int64)
    cpu["start"], dev["start"] = start, torch.tensor(start, device="cuda")
    _, logp, d = policy(g, x, host, dev, cpu, mean="sequence")
    assert not d[:5].any() and not d[690:].any()


def test_gradients_against_differences(g):
    """The device's own loss along a direction: central differences at step h of fp32 losses.

    Rounding: each loss carries at most 2e-7 times the mean magnitude of its
    terms (below 4), over 2h; truncation h^2 / 6 times a third derivative along
    v, |v|_inf <= 1, below 30: 1e-4 + 3e-3 at h = 0.025."""
    x, _, dev, _ = make(24, 50, torch.float32, seed=11, n_seq=4, masked=0.2, spread=1.0)
    # ratios close to 1: the differences do not cross the clip's edges
    now = g.ar_token_logp(x, dev["labels"])
    dev["old"] = now - 0.02
    v = torch.randn(24, 50, generator=torch.Generator().manual_seed(1)).cuda().clamp(-1, 1)
    h = 0.025

    def pol(y, **kw):
        return g.ar_policy_loss(y, dev["labels"], dev["old"], dev["adv"], dev["start"], ref_logp=dev["ref"],
                                kl_coef=0.2, **kw)

    def pref(y, **kw):
        return g.ar_preference_loss(y, dev["labels"], dev["ref"], dev["start"], beta=0.5, **kw)

    for f in (pol, pref):
        grad = f(x)[-1]
        want = float(f(x + h * v, grad=False)[0][0] - f(x - h * v, grad=False)[0][0]) / (2 * h)
        got = float((grad.double() * v.double()).sum())
        assert abs(got - want) < 3.2e-3 and abs(got) > 1e-2, (got, want)


def test_repeatable_and_on_another_stream(g):
    x, host, dev, cpu = make(300, 3001, torch.bfloat16, seed=6, n_seq=8)
    a = policy(g, x, host, dev, cpu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [g.ar_policy_loss(x, dev["labels"], dev["old"], dev["adv"], dev["start"], ref_logp=dev["ref"],
                                 clip_low=CLIP[0], clip_high=CLIP[1], kl_coef=0.1) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    for b in outs:
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_in_a_graph(g):
    x, host, dev, cpu = make(40, 999, torch.float32, seed=7, n_seq=4)
    want = preference(g, x, host, dev, cpu)
    ws = torch.empty(g.ar_loss_workspace(40, 4), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.ar_preference_loss(x, dev["labels"], dev["ref"], dev["start"], stats=outs[0], ratios=outs[1], logp=outs[2],
                             dlogits=outs[3], workspace=ws)
    for _ in range(2):
        for o in outs:
            o.fill_(5.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs, want))


def test_offsets_beyond_32_bits(g):
    """Rows whose element offsets pass 2^31 (bf16, 13 GB of address range)."""
    ld, vocab = (1 << 31) + 24, 1000
    flat = torch.empty(2 * ld + vocab, dtype=torch.bfloat16, device="cuda")
    x, host, dev, cpu = make(3, vocab, torch.bfloat16, seed=1, masked=0.0)
    far = flat.as_strided((3, vocab), (ld, 1))
    far.copy_(x)
    near = policy(g, x, host, dev, cpu)
    got = policy(g, far, host, dev, cpu, dlogits=far)
    assert all(torch.equal(a, b) for a, b in zip(near, got))
