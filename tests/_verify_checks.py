"""Inputs for the verification of drafted tokens, with no decision on its edge, and the check of a call."""

import numpy as np
import torch

from oracle import verify as V


def make(counts, vocab, dtype="f32", seed=0, drafted=True, temperature=1.0, spread=2.0, blur=0.8, ruled=0.0,
         draft_dtype=None):
    """dict of target, drafts, uniforms, draft_start, draft_logits (host tensors)."""
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    n, rows = int(start[-1]), int(start[-1]) + len(counts)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    target = rng.normal(size=(rows, vocab)) * spread
    if ruled:
        out = rng.random(vocab) < ruled
        out[0] = False
        target[:, out] = -np.inf
    target = torch.from_numpy(target).to(kind[dtype])
    which = np.repeat(np.arange(len(counts)), counts)
    at = torch.from_numpy(np.arange(n) + which)
    draft_logits = None
    drafts = np.zeros(n, np.int64)
    if drafted:
        draft_logits = (target[at].double() + blur * torch.from_numpy(rng.normal(size=(n, vocab)))).to(
            kind[draft_dtype or dtype])
    for i in range(n):
        q = V.softmax((draft_logits if drafted else target[at])[i].double().numpy(), temperature)
        drafts[i] = rng.choice(vocab, p=q) if rng.random() < 0.7 or drafted else int(np.argmax(q))
    return dict(target=target, drafts=torch.from_numpy(drafts), uniforms=torch.from_numpy(rng.random(rows).astype(np.float32)),
                draft_start=torch.from_numpy(start), draft_logits=draft_logits)


def want(c, temperature=1.0, greedy=False, draft_temperature=None):
    wide = [None if c[k] is None else c[k].double().numpy() for k in ("target", "draft_logits")]
    return V.verify(wide[0], c["drafts"].numpy(), c["uniforms"].double().numpy(), c["draft_start"].tolist(), wide[1],
                    temperature, draft_temperature, greedy)


# What a decision may be off by. A ratio p/q is the exponential of a difference of log-probabilities, each the sum of
# a product in 64 bits and a logarithm that carries the fp32 error of a sum of exponentials: their arguments are
# rounded to 2^-24 of up to 2^5 in base 2, the exponential itself to 2^-22: below 2^-18. A running sum's terms
# are off by 2^-21 of themselves, so that sums and total are off by 2^-20 of what was summed: p and q, at most 2.
RATIO, SUM = 2.0 ** -16, 2.0 ** -18


def settle(c, temperature=1.0, draft_temperature=None):
    """Moves uniform numbers off the edges of decisions: every decision that is made has more room than rounding
    could take (most already have)."""
    for _ in range(8):
        accepted, tokens, _, margins = want(c, temperature, False, draft_temperature)
        start = c["draft_start"].tolist()
        finals = {start[s + 1] + s for s in range(len(start) - 1)}
        bad = [r for r in range(len(margins)) if margins[r] < (SUM if r in finals else RATIO)]
        if not bad:
            return accepted, tokens, margins
        for r in bad:
            c["uniforms"][r] = float(c["uniforms"][r]) * 0.983 + 0.004
    raise AssertionError("inputs without room")


def call(g, c, temperature=1.0, mode="sample", device="cuda", **kw):
    d = {k: None if v is None else v.to(device) for k, v in c.items()}
    if mode == "greedy":
        d["uniforms"] = None
    return g.ar_verify_drafts(d["target"], d["drafts"], d["uniforms"], d["draft_start"], draft_logits=d["draft_logits"],
                              temperature=temperature, mode=mode, **kw)


def check(got, expected, where=""):
    accepted, tokens, logp = (t.cpu().numpy() for t in got)
    assert np.array_equal(accepted, expected[0]), (where, accepted, expected[0])
    assert np.array_equal(tokens, expected[1]), (where, np.nonzero(tokens != expected[1]))
    # a log-probability: the fp32 error of the sum's exponentials (2^-19 of it, as above), and its own rounding
    room = 2.0 ** -19 + np.abs(expected[2]) * 2.0 ** -23
    assert np.array_equal(np.isnan(logp), np.isnan(expected[2])), where
    assert (np.abs(logp - expected[2])[~np.isnan(logp)] <= room[~np.isnan(logp)]).all(), (where, np.abs(logp - expected[2]).max())
