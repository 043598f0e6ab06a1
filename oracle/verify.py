"""Verification of drafted tokens in 64 bits, from its definition (numpy), token by token. No code
is shared with the GPU path."""

from __future__ import annotations

import numpy as np

FALL, STAND = 0, 1


def softmax(x, temperature=1.0):
    """Probabilities of a row, None where it is no distribution."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
        return None
    e = np.exp((x - x.max()) / temperature)
    return e / e.sum()


def residue(p, q):
    """What a token is drawn from behind a draft that fell: max(p - q, 0), or p where that is nothing."""
    w = np.maximum(p - q, 0.0)
    return w if w.sum() > 0 else p


def draw(w, u):
    """The first index whose running sum passes u times the total."""
    upto = np.cumsum(w)
    return int(np.searchsorted(upto, min(max(u, 0.0), 1.0) * upto[-1], side="right"))


def verify(target, drafts, uniforms, draft_start, draft_logits=None, temperature=1.0, draft_temperature=None,
           greedy=False):
    """(accepted, tokens, logp, margins): margins[r] is how far row r's decision is from the next other one:
    |u - p/q| / (p/q) for a draft; for a drawn token, the distance of u to the ends of its share of the total,
    times the total."""
    target = np.asarray(target, np.float64)
    rows, vocab = target.shape
    tokens, logp, margins = np.full(rows, -1), np.zeros(rows), np.full(rows, np.inf)
    accepted = []
    for s in range(len(draft_start) - 1):
        first, count = draft_start[s], draft_start[s + 1] - draft_start[s]
        for j in range(count + 1):
            row = first + s + j
            x = int(drafts[first + j]) if j < count else -1
            p = softmax(target[row], temperature)
            q = np.zeros(vocab)
            if j < count and draft_logits is not None:
                q = softmax(draft_logits[first + j], draft_temperature or temperature)
            elif 0 <= x < vocab:
                q[x] = 1.0
            if p is None or q is None:
                logp[row] = np.nan
                accepted.append(j)
                break
            if greedy:
                token = int(np.argmax(target[row]))
                stands = token == x
            else:
                stands = False
                if 0 <= x < vocab and p[x] > 0:
                    ratio = p[x] / q[x] if q[x] > 0 else np.inf
                    stands = uniforms[row] < ratio
                    if np.isfinite(ratio):
                        margins[row] = abs(uniforms[row] - ratio) / ratio
                if not stands:
                    w = p if j == count else residue(p, q)
                    u = float(uniforms[first + count + s])
                    token = draw(w, u)
                    upto = np.cumsum(w)
                    at = u * upto[-1]
                    margins[first + count + s] = min(margins[first + count + s], upto[token] - at,
                                                     at - (upto[token] - w[token]) if token else np.inf)
            if stands:
                tokens[row], logp[row] = x, np.log(p[x])
                continue
            tokens[row], logp[row] = token, np.log(p[token])
            accepted.append(j)
            break
    return np.array(accepted), tokens, logp, margins


def emitted(p, q):
    """The distribution of one token from a draft of q verified against p: drafts that stand, and draws behind
    those that fall. It is p."""
    stands = np.minimum(p, q)
    return stands + (1.0 - stands.sum()) * residue(p, q) / residue(p, q).sum()
