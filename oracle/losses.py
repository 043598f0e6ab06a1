"""The losses on a language model's logits and their gradients, in 64 bits, from
their formulas (numpy). Row by row, sequence by sequence; no code is shared with
the GPU path.

Every function takes logits [rows, vocab] (any float type, widened exactly),
integer labels (negative: the row is not part of the loss) and a temperature.
"""

from __future__ import annotations

import numpy as np


def log_softmax(logits, temperature=1.0):
    x = np.asarray(logits, np.float64) / temperature
    with np.errstate(invalid="ignore", divide="ignore"):
        x = x - x.max(axis=1, keepdims=True)
        return x - np.log(np.exp(x).sum(axis=1, keepdims=True))


def token_logp(logits, labels, temperature=1.0):
    """Log-probabilities of the labels; 0 where a label is negative."""
    labels = np.asarray(labels)
    out = np.zeros(len(labels))
    rows = np.nonzero(labels >= 0)[0]
    if rows.size:
        out[rows] = log_softmax(np.asarray(logits)[rows], temperature)[np.arange(rows.size), labels[rows]]
    return out


def logits_gradient(logits, labels, slope, temperature=1.0):
    """slope[t] * (onehot(label) - softmax) / temperature; zeros where a label is negative."""
    logits = np.asarray(logits)
    out = np.zeros(logits.shape)
    for t, y in enumerate(labels):
        if y < 0 or slope[t] == 0.0:
            continue
        p = np.exp(log_softmax(logits[t:t + 1], temperature)[0])
        p = -p
        p[y] += 1.0
        out[t] = slope[t] / temperature * p
    return out


def weights(labels, seq_start, mean="token", denominator=0.0):
    """Each row's weight in the mean over labelled tokens, or over sequences of such means."""
    labels = np.asarray(labels)
    counted = np.zeros(len(labels))
    total = 0
    for lo, hi in zip(seq_start[:-1], seq_start[1:]):
        n = int((labels[lo:hi] >= 0).sum())
        if n == 0:
            continue
        total += n if mean == "token" else 1
        counted[lo:hi] = np.where(labels[lo:hi] >= 0, 1.0 if mean == "token" else 1.0 / n, 0.0)
    return counted / (denominator if denominator > 0 else max(total, 1))


def policy_from_logp(logp, old, adv, w, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0):
    """(stats, slope): the loss's statistics and dL/dlogp."""
    logp, old, adv = (np.asarray(v, np.float64) for v in (logp, old, adv))
    stats, slope = np.zeros(4), np.zeros(len(logp))
    for t in np.nonzero(w)[0]:
        r = np.exp(logp[t] - old[t])
        free, held = r * adv[t], min(max(r, 1 - clip_low), 1 + clip_high) * adv[t]
        stats[1] += w[t] * -min(free, held)
        stats[3] += w[t] * (held < free)
        if free <= held:
            slope[t] -= w[t] * free
        if ref is not None:
            b = float(ref[t]) - logp[t]
            stats[2] += w[t] * (np.exp(b) - b - 1)
            slope[t] += w[t] * kl_coef * (1 - np.exp(b))
    stats[0] = stats[1] + kl_coef * stats[2]
    return stats, slope


def policy_loss(logits, labels, old, adv, seq_start, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                temperature=1.0, mean="token", denominator=0.0, grad_scale=1.0):
    """dict of stats, logp, dlogits, slope (dL/dlogp times grad_scale)."""
    logp = token_logp(logits, labels, temperature)
    w = weights(labels, seq_start, mean, denominator)
    stats, slope = policy_from_logp(logp, old, adv, w, ref, clip_low, clip_high, kl_coef)
    slope = slope * grad_scale
    return dict(stats=stats, logp=logp, slope=slope, weights=w,
                dlogits=logits_gradient(logits, labels, slope, temperature))


def preference_from_logp(logp, labels, ref, seq_start, beta=0.1, form="sigmoid", label_smoothing=0.0, target=0.5,
                         length_normalized=False, denominator=0.0):
    """(stats, ratios, slope): statistics, log ratios of the sequences, dL/dlogp."""
    labels = np.asarray(labels)
    n_seq = len(seq_start) - 1
    ratios, over = np.zeros(n_seq), np.ones(n_seq)
    for s in range(n_seq):
        rows = [t for t in range(seq_start[s], seq_start[s + 1]) if labels[t] >= 0]
        if length_normalized:
            over[s] = max(len(rows), 1)
        ratios[s] = sum(float(logp[t]) - float(ref[t]) for t in rows) / over[s]
    pairs = n_seq // 2
    count = denominator if denominator > 0 else pairs
    stats, slope = np.zeros(4), np.zeros(len(labels))
    for i in range(pairs):
        good, bad = ratios[2 * i], ratios[2 * i + 1]
        z = beta * (good - bad)
        if form == "sigmoid":
            loss = (1 - label_smoothing) * np.logaddexp(0, -z) + label_smoothing * np.logaddexp(0, z)
            dz = -(1 - label_smoothing) / (1 + np.exp(z)) + label_smoothing / (1 + np.exp(-z))
        else:
            loss, dz = (z - target) ** 2, 2 * (z - target)
        stats += np.array([loss, beta * good, beta * bad, float(good > bad)]) / count
        for s, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            for t in range(seq_start[s], seq_start[s + 1]):
                if labels[t] >= 0:
                    slope[t] = sign * dz * beta / count / over[s]
    return stats, ratios, slope


def preference_loss(logits, labels, ref, seq_start, temperature=1.0, grad_scale=1.0, **kw):
    """dict of stats, ratios, logp, dlogits, slope (dL/dlogp times grad_scale)."""
    logp = token_logp(logits, labels, temperature)
    stats, ratios, slope = preference_from_logp(logp, labels, ref, seq_start, **kw)
    slope = slope * grad_scale
    return dict(stats=stats, ratios=ratios, logp=logp, slope=slope,
                dlogits=logits_gradient(logits, labels, slope, temperature))
