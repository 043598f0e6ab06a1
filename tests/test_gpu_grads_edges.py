"""Calls of the gradient operators with some outputs in place and some elsewhere."""

import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
SHAPES = [(100,), (4097,), (33,), (0,), (9000,)]
NAMES = ("params", "exp_avgs", "exp_avg_sqs", "masters")


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def adam_state(seed, masters, param=torch.bfloat16):
    """Lists by name; a parameter beside a master is that one, rounded. `masters`: which tensors have one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal():
        return [torch.randn(s, generator=gen, device="cuda") for s in SHAPES]

    s = dict(masters=[w if m else None for w, m in zip(normal(), masters)], exp_avgs=normal(),
             exp_avg_sqs=[v.square() for v in normal()])
    s["params"] = [(p if w is None else w).to(param) for p, w in zip(normal(), s["masters"])]
    return s, normal()


@pytest.mark.parametrize("elsewhere", [c for n in range(5) for c in itertools.combinations(NAMES, n)],
                         ids=lambda c: "+".join(c) or "none")
@pytest.mark.parametrize("masters", [(True,) * 5, (True, False, True, True, False)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_skipped_step_writes_every_output_that_is_elsewhere(g, elsewhere, masters, bad):
    s, grads = adam_state(1, masters)
    keep = {k: [None if t is None else t.clone() for t in v] for k, v in s.items()}
    grads[1][4000] = bad
    stats, _ = g.ar_grad_norm(grads, 1.0)
    outs = {k: [None if t is None else torch.full_like(t, float("nan")) for t in s[k]] for k in elsewhere}
    g.ar_adamw_step(s["params"], grads, s["exp_avgs"], s["exp_avg_sqs"], 0.1, 3, weight_decay=0.1, clip=stats,
                    masters=s["masters"], **{k + "_out": v for k, v in outs.items()})
    for k in NAMES:
        for before, now, out in zip(keep[k], s[k], outs.get(k, s[k])):
            assert before is None or (torch.equal(now, before) and torch.equal(out, before)), k


@pytest.mark.parametrize("elsewhere", [("params",), ("masters",), ("exp_avgs",), ("params", "masters")])
def test_a_step_with_some_outputs_elsewhere(g, elsewhere):
    """The same bits as in place; inputs whose outputs are elsewhere stay."""
    s, grads = adam_state(2, (True, False, True, True, False))
    keep = {k: [None if t is None else t.clone() for t in v] for k, v in s.items()}
    same = {k: [None if t is None else t.clone() for t in v] for k, v in s.items()}
    stats, _ = g.ar_grad_norm(grads, 1.0)

    def step(x, **outs):
        g.ar_adamw_step(x["params"], grads, x["exp_avgs"], x["exp_avg_sqs"], 0.1, 3, weight_decay=0.1, clip=stats,
                        masters=x["masters"], **outs)

    step(same)
    outs = {k: [None if t is None else torch.full_like(t, float("nan")) for t in s[k]] for k in elsewhere}
    step(s, **{k + "_out": v for k, v in outs.items()})
    for k in NAMES:
        for before, now, out, want in zip(keep[k], s[k], outs.get(k, s[k]), same[k]):
            assert before is None or torch.equal(out, want), k
            assert before is None or k not in elsewhere or torch.equal(now, before), k
