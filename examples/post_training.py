"""A data-parallel post-training step over N virtual ranks, from logits to weights.

Each rank samples answers from a small policy, scores them, and differentiates
a loss on its own answers; the gradients of all ranks are summed bucket by
bucket, and the orthogonalised step updates the weights:

    ar_verify_drafts                  with --drafts: tokens drafted by the reference policy, kept or redrawn
    ar_token_logp                     log-probabilities under the old and the reference policy
    ar_policy_loss / ar_preference_loss  the loss and the gradient of the logits, in one call
    BucketedReducer                   the sum over the ranks' gradients
    ar_grad_norm                      with --max-norm: the global norm, whose coefficient the steps read
    ar_muon_step                      momentum, orthogonalisation, weight update
    ar_adamw_step                     with --adamw: the step of embedding and head

    python examples/post_training.py [--objective policy|preference] [--steps 12] [--ranks 4]
                                     [--drafts 0] [--max-norm X] [--adamw]

The policy is a one-hidden-layer model of the next token given the last one;
an answer's reward is the share of its tokens below vocab / 2.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_sync_gb300 as g  # noqa: E402
from gradient_sync_gb300.overlap import BucketedReducer  # noqa: E402


class Policy:
    """logits = head(relu(up(embedding[token]))), fp32 weights."""

    def __init__(self, vocab, hidden, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols, fan_in):
            return torch.randn(rows, cols, generator=gen, device="cuda") / fan_in ** 0.5

        self.weights = [weight(vocab, hidden, 1), weight(2 * hidden, hidden, hidden),
                        weight(vocab, 2 * hidden, 2 * hidden)]

    def logits(self, tokens, weights=None):
        embedding, up, head = weights or self.weights
        return torch.relu(embedding[tokens] @ up.T) @ head.T


def rollouts(policy, answers, length, vocab, gen):
    """(tokens before, tokens after, offsets): answers of 1..length tokens, sampled one token at a time."""
    last = torch.randint(0, vocab, (answers,), generator=gen, device="cuda")
    before, after = [], []
    for _ in range(length):
        p = torch.softmax(policy.logits(last), 1)
        nxt = torch.multinomial(p, 1, generator=gen)[:, 0]
        before.append(last)
        after.append(nxt)
        last = nxt
    lengths = torch.randint(1, length + 1, (answers,), generator=gen, device="cuda")
    keep = torch.arange(length, device="cuda")[None, :] < lengths[:, None]
    start = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])
    return torch.stack(before, 1)[keep], torch.stack(after, 1)[keep], start


def drafted_rollouts(policy, draft, answers, length, vocab, gen, drafts):
    """The same, `drafts` tokens at a time: drafted by the policy `draft`, verified by one pass of `policy`. Also the
    tokens' log-probabilities under it."""
    rows = torch.arange(answers, device="cuda")
    last = torch.randint(0, vocab, (answers,), generator=gen, device="cuda")
    have = torch.zeros_like(last)
    room = length + drafts + 1
    before, after = torch.zeros(2, answers, room, dtype=torch.long, device="cuda")
    logps = torch.zeros(answers, room, device="cuda")
    starts = torch.arange(answers + 1, device="cuda") * drafts
    place = torch.arange(drafts + 1, device="cuda")
    while int(have.min()) < length:
        chain, scores = [last], []
        for _ in range(drafts):
            scores.append(draft.logits(chain[-1]))
            chain.append(torch.multinomial(torch.softmax(scores[-1], 1), 1, generator=gen)[:, 0])
        chain = torch.stack(chain, 1)
        u = torch.rand(answers * (drafts + 1), generator=gen, device="cuda")
        kept, tokens, logp = g.ar_verify_drafts(
            policy.logits(chain.reshape(-1)), chain[:, 1:].contiguous().reshape(-1), u, starts,
            draft_logits=torch.stack(scores, 1).reshape(answers * drafts, vocab))
        tokens, logp = tokens.reshape(answers, -1), logp.reshape(answers, -1)
        at = (have[:, None] + place).clamp(max=room - 1)
        fits = (place <= kept[:, None]) & (at < length)
        at = torch.where(fits, at, torch.full_like(at, room - 1))  # (the last place is nobody's)
        before.scatter_(1, at, torch.where(place == 0, last[:, None], tokens.roll(1, 1)))
        after.scatter_(1, at, tokens)
        logps.scatter_(1, at, logp)
        have = (have + kept + 1).clamp(max=length)
        last = tokens[rows, kept]
    lengths = torch.randint(1, length + 1, (answers,), generator=gen, device="cuda")
    keep = torch.arange(room, device="cuda")[None, :] < lengths[:, None]
    start = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])
    return before[keep], after[keep], start, logps[keep]


def sequence_means(values, start):
    total = torch.cat([values.new_zeros(1), values.cumsum(0)])
    return (total[start[1:]] - total[start[:-1]]) / (start[1:] - start[:-1])


def train(objective="policy", steps=12, ranks=4, answers=64, length=24, vocab=512, hidden=128, lr=0.2, seed=0,
          drafts=0, max_norm=None, adamw=False):
    """Runs `steps` steps; returns the mean reward of the ranks' answers at each."""
    policy, frozen = Policy(vocab, hidden, seed), Policy(vocab, hidden, seed)
    reference = frozen.weights
    matrices, others = ([1], [0, 2]) if adamw else ([0, 1, 2], [])

    def of(which, tensors):
        return [tensors[i] for i in which]

    momenta = [torch.zeros_like(w) for w in of(matrices, policy.weights)]
    moments = [[torch.zeros_like(w) for w in of(others, policy.weights)] for _ in range(2)]
    updates = 0
    plan = g.ar_ortho_plan([tuple(w.shape) for w in of(matrices, policy.weights)])
    workspace = torch.empty(g.ar_ortho_workspace(plan), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    rewards = []
    for _ in range(steps):
        batches = []
        for _ in range(ranks):
            old = None
            if drafts:
                before, after, start, old = drafted_rollouts(policy, frozen, answers, length, vocab, gen, drafts)
            else:
                before, after, start = rollouts(policy, answers, length, vocab, gen)
            score = sequence_means((after < vocab // 2).float(), start)
            if objective == "preference":  # the better of two answers first
                first = (score[0::2] < score[1::2]).long() + torch.arange(0, answers, 2, device="cuda")
                order = torch.stack([first, torch.arange(0, answers, 2, device="cuda") * 2 + 1 - first], 1).reshape(-1)
                spans = [torch.arange(int(start[i]), int(start[i + 1]), device="cuda") for i in order.tolist()]
                rows = torch.cat(spans)
                start = torch.tensor([0] + [len(s) for s in spans], device="cuda").cumsum(0)
                before, after, score = before[rows], after[rows], score[order]
                old = None
            with torch.no_grad():
                old = g.ar_token_logp(policy.logits(before), after) if old is None else old
                ref = g.ar_token_logp(policy.logits(before, reference), after)
            which = torch.repeat_interleave(torch.arange(answers, device="cuda"), start[1:] - start[:-1])
            advantage = (score - score.mean()) / (score.std() + 1e-6)
            batches.append((before, after, start, old, ref, advantage[which].contiguous()))
            rewards_now = score.mean() if len(batches) == 1 else rewards_now + score.mean()
        rewards.append(float(rewards_now) / ranks)
        tokens = sum(len(b[0]) for b in batches)
        for _ in range(2 if objective == "policy" else 1):  # updates on the same answers
            grads = []
            for before, after, start, old, ref, advantage in batches:
                weights = [w.detach().requires_grad_() for w in policy.weights]
                logits = policy.logits(before, weights)
                x = logits.detach()
                # the mean is over all ranks: their gradients are summed as they are
                if objective == "policy":
                    d = g.ar_policy_loss(x, after, old, advantage, start, ref_logp=ref, kl_coef=0.01,
                                         denominator=tokens)[2]
                else:
                    d = g.ar_preference_loss(x, after, ref, start, beta=0.2, denominator=ranks * answers // 2)[3]
                grads.append(list(torch.autograd.grad(logits, weights, d)))
            reducer = BucketedReducer(grads, scale=1.0)
            for t in reversed(range(len(policy.weights))):
                reducer.ready(t)
            reducer.finish()
            clip = None if max_norm is None else g.ar_grad_norm(grads[0], max_norm)[0]
            g.ar_muon_step(plan, of(matrices, policy.weights), of(matrices, grads[0]), momenta, lr=lr,
                           workspace=workspace, clip=clip)
            updates += 1
            if others:
                g.ar_adamw_step(of(others, policy.weights), of(others, grads[0]), *moments, lr=0.1 * lr, step=updates,
                                clip=clip)
    return rewards


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--objective", choices=("policy", "preference"), default="policy")
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=0, help="tokens that the reference policy drafts at a time")
    ap.add_argument("--max-norm", type=float, help="clip the gradients' global norm")
    ap.add_argument("--adamw", action="store_true", help="embedding and head take AdamW steps")
    a = ap.parse_args(argv)
    for i, r in enumerate(train(a.objective, a.steps, a.ranks, drafts=a.drafts, max_norm=a.max_norm, adamw=a.adamw)):
        print(f"step {i}: mean reward {r:.3f}")


if __name__ == "__main__":
    main()
