"""Refusals of the losses' entry points, without a GPU: every bad argument is
answered before any device work is enqueued."""

import ctypes

import pytest

A = 1 << 20  # a stand-in device address: the calls below return before it is used


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def logits(g, **kw):
    d = dict(data=A, rows=4, vocab=10, ld=10, dtype=g.AR_F32, labels=2 * A, temperature=1.0)
    d.update(kw)
    return g._lib.ArLogits(*[d[f] for f, _ in g._lib.ArLogits._fields_])


BAD_LOGITS = [dict(rows=-1), dict(vocab=0), dict(ld=9), dict(dtype=7), dict(temperature=0.0), dict(temperature=-1.0),
              dict(temperature=float("nan")), dict(temperature=float("inf")), dict(temperature=1e-45), dict(data=0),
              dict(data=A + 2), dict(dtype=1, data=A + 1), dict(labels=0), dict(labels=A + 4),
              dict(rows=1 << 30, ld=1 << 40)]


@pytest.mark.parametrize("bad", BAD_LOGITS)
def test_bad_logits(g, bad):
    lib = g._lib.load()
    x = logits(g, **bad)
    assert lib.ar_token_logp(x, 3 * A, None) == g.AR_EINVAL
    assert policy(g, x) == g.AR_EINVAL
    assert preference(g, x) == g.AR_EINVAL


def test_logp_outputs(g):
    lib = g._lib.load()
    assert lib.ar_token_logp(None, 3 * A, None) == g.AR_EINVAL
    assert lib.ar_token_logp(logits(g), 0, None) == g.AR_EINVAL
    assert lib.ar_token_logp(logits(g), 3 * A + 2, None) == g.AR_EINVAL
    assert lib.ar_token_logp(logits(g), A + 8, None) == g.AR_EINVAL      # inside the logits
    assert lib.ar_token_logp(logits(g), 2 * A + 8, None) == g.AR_EINVAL  # inside the labels
    assert lib.ar_token_logp(logits(g, rows=1 << 31), 3 * A, None) == g.AR_EUNSUPPORTED


def policy(g, x=None, desc=None, **kw):
    a = dict(old=3 * A, ref=4 * A, adv=5 * A, start=6 * A, n_seq=2, stats=7 * A, logp=8 * A, d=9 * A, dld=10,
             ws=10 * A)
    a.update(kw)
    d = dict(clip_low=0.2, clip_high=0.2, kl_coef=0.1, mean=0, denominator=0.0, grad_scale=1.0)
    d.update(desc or {})
    return g._lib.load().ar_policy_loss(x if x is not None else logits(g), a["old"], a["ref"], a["adv"], a["start"],
                                        a["n_seq"], g._lib.ArPolicyDesc(*d.values()), a["stats"], a["logp"], a["d"],
                                        a["dld"], a["ws"], None)


@pytest.mark.parametrize("bad", [dict(old=0), dict(old=3 * A + 1), dict(adv=0), dict(ref=0), dict(ref=4 * A + 2),
                                 dict(start=0), dict(start=6 * A + 4), dict(n_seq=0), dict(n_seq=-3), dict(stats=0),
                                 dict(logp=0), dict(logp=8 * A + 1), dict(dld=9), dict(d=9 * A + 2), dict(ws=0),
                                 dict(ws=10 * A + 8), dict(d=A + 40), dict(d=A, dld=12), dict(logp=3 * A + 4),
                                 dict(stats=8 * A), dict(ws=9 * A), dict(stats=A)])
def test_policy_refusals(g, bad):
    assert policy(g, **bad) == g.AR_EINVAL


@pytest.mark.parametrize("bad", [dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-1.0),
                                 dict(clip_high=float("inf")), dict(kl_coef=-1.0), dict(kl_coef=float("nan")),
                                 dict(mean=2), dict(denominator=-1.0), dict(denominator=float("nan")),
                                 dict(grad_scale=float("inf"))])
def test_policy_descriptor_refusals(g, bad):
    assert policy(g, desc=bad) == g.AR_EINVAL


def preference(g, x=None, desc=None, **kw):
    a = dict(ref=4 * A, start=6 * A, n_seq=2, stats=7 * A, ratios=5 * A, logp=8 * A, d=9 * A, dld=10, ws=10 * A)
    a.update(kw)
    d = dict(beta=0.1, form=0, label_smoothing=0.0, target=0.5, length_normalized=0, denominator=0.0, grad_scale=1.0)
    d.update(desc or {})
    return g._lib.load().ar_preference_loss(x if x is not None else logits(g), a["ref"], a["start"], a["n_seq"],
                                            g._lib.ArPreferenceDesc(*d.values()), a["stats"], a["ratios"], a["logp"],
                                            a["d"], a["dld"], a["ws"], None)


@pytest.mark.parametrize("bad", [dict(ref=0), dict(start=0), dict(n_seq=3), dict(n_seq=0), dict(stats=0),
                                 dict(ratios=0), dict(ratios=8 * A), dict(logp=0), dict(dld=9), dict(ws=0),
                                 dict(d=A + 4), dict(d=4 * A)])
def test_preference_refusals(g, bad):
    assert preference(g, **bad) == g.AR_EINVAL


@pytest.mark.parametrize("bad", [dict(beta=float("nan")), dict(form=2), dict(label_smoothing=0.6),
                                 dict(label_smoothing=-0.1), dict(target=float("inf")), dict(denominator=-2.0)])
def test_preference_descriptor_refusals(g, bad):
    assert preference(g, desc=bad) == g.AR_EINVAL


def test_workspace_size(g):
    b = ctypes.c_size_t()
    lib = g._lib.load()
    assert lib.ar_loss_workspace(0, 0, b) == g.AR_OK and b.value >= 256
    assert lib.ar_loss_workspace(-1, 0, b) == g.AR_EINVAL
    assert lib.ar_loss_workspace(1, -1, b) == g.AR_EINVAL
    assert lib.ar_loss_workspace(1, 1, None) == g.AR_EINVAL
    assert g.ar_loss_workspace(1000, 10) > g.ar_loss_workspace(10, 10)


def test_binding_refuses_other_tensors(g):
    import torch

    x, y = torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        g.ar_token_logp(x, y)  # not on a GPU
