"""The orthogonalised step with the clipping coefficient of a gradient norm: as after clipping, without a pass of its own."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
SHAPES = [(64, 96), (130, 70), (1, 33), (33, 129)]


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def state(dtype="f32", seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    return ([torch.randn(s, generator=gen, device="cuda").to(kind) for s in SHAPES],
            [torch.randn(s, generator=gen, device="cuda").to(kind) for s in SHAPES],
            [torch.randn(s, generator=gen, device="cuda") for s in SHAPES])


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("precision", ["half", "split"])
def test_as_after_clipping(g, nesterov, precision):
    """fp32 gradients: clipping them first rounds the same product, so that the two give equal bits."""
    w, grads, m = state()
    plan = g.ar_ortho_plan(SHAPES, precision=precision)
    stats, _, clipped = g.ar_grad_clip(grads, 0.7, outs=[torch.empty_like(x) for x in grads])
    assert stats[2] == 1.0
    a, b = [[x.clone() for x in v] for v in (w, m)], [[x.clone() for x in v] for v in (w, m)]
    g.ar_muon_step(plan, a[0], clipped, a[1], lr=0.1, weight_decay=0.1, nesterov=nesterov)
    g.ar_muon_step(plan, b[0], grads, b[1], lr=0.1, weight_decay=0.1, nesterov=nesterov, clip=stats)
    for x, y in zip(a, b):
        assert all(torch.equal(p, q) for p, q in zip(x, y))
    # where nothing is clipped, the step without
    stats, _ = g.ar_grad_norm(grads, 1e9, grad_scale=0.5)
    a, b = [[x.clone() for x in v] for v in (w, m)], [[x.clone() for x in v] for v in (w, m)]
    g.ar_muon_step(plan, a[0], grads, a[1], lr=0.1, grad_scale=0.5, nesterov=nesterov)
    g.ar_muon_step(plan, b[0], grads, b[1], lr=0.1, grad_scale=0.5, nesterov=nesterov, clip=stats)
    for x, y in zip(a, b):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("nesterov", [False, True])
def test_gradients_that_are_not_finite_count_as_zero(g, dtype, bad, nesterov):
    w, grads, m = state(dtype)
    grads[1][3, 5] = bad
    plan = g.ar_ortho_plan(SHAPES, dtype, dtype)
    stats, _ = g.ar_grad_norm(grads, 1.0)
    a, b = [[x.clone() for x in v] for v in (w, m)], [[x.clone() for x in v] for v in (w, m)]
    g.ar_muon_step(plan, a[0], grads, a[1], lr=0.1, nesterov=nesterov, clip=stats)
    g.ar_muon_step(plan, b[0], [torch.zeros_like(x) for x in grads], b[1], lr=0.1, nesterov=nesterov)
    for x, y in zip(a, b):
        assert all(torch.equal(p, q) and p.isfinite().all() for p, q in zip(x, y))


def test_momentum_against_the_formula(g):
    """M' = mu M + c s G, three fp32 roundings; bf16 gradients, scaled in fp32."""
    w, grads, m = state("bf16", 3)
    plan = g.ar_ortho_plan(SHAPES, "bf16", "bf16")
    stats, _ = g.ar_grad_norm(grads, 0.3, grad_scale=0.25)
    new = [torch.empty_like(x) for x in m]
    g.ar_muon_step(plan, w, grads, m, lr=0.1, momentum=0.9, grad_scale=0.25, clip=stats, momenta_out=new)
    c = float(stats[1]) * 0.25
    for x, y, z in zip(new, m, grads):
        want = 0.9 * y.double() + c * z.double()
        # mu in fp32, the factor, the product, the sum
        room = 2.0 ** -24 * (2 * (0.9 * y.double()).abs() + 3 * (c * z.double()).abs() + want.abs())
        assert ((x.double() - want).abs() <= room).all()


def test_whole_step_in_a_graph(g):
    """One norm over all gradients, the matrices' step and the others' AdamW step reading it, captured and replayed."""
    w, grads, m = state(seed=5)
    gains, dgains = torch.randn(500, device="cuda"), torch.randn(500, device="cuda")
    ms, vs, t = torch.zeros(500, device="cuda"), torch.zeros(500, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    plan = g.ar_ortho_plan(SHAPES)
    one = torch.ones_like(t)

    def step():
        t.add_(one)
        stats, _ = g.ar_grad_norm([*grads, dgains], 1.0)
        g.ar_muon_step(plan, w, grads, m, lr=0.02, clip=stats)
        g.ar_adamw_step([gains], [dgains], [ms], [vs], 1e-2, t, clip=stats)

    state_ = [*w, *m, gains, ms, vs, t]
    start = [x.clone() for x in state_]
    for _ in range(3):
        step()
    want = [x.clone() for x in state_]
    for x, y in zip(state_, start):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip(state_, start):
        x.copy_(y)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(state_, want))
    assert g.ar_device_status() == g.AR_OK
