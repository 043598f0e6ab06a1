"""What the steps behind a norm do with gradients that are not finite: AdamW skips its step, the orthogonalised step goes on
along its old momentum, and so do steps that are given a clipping call's zeros."""

import pytest
import torch

pytestmark = pytest.mark.gpu
SHAPES = [(64, 96), (130, 70), (33, 129)]


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


@pytest.fixture(params=[float("nan"), float("inf")])
def bad(request):
    gen = torch.Generator(device="cuda").manual_seed(1)
    w, grads, m = ([torch.randn(s, generator=gen, device="cuda") for s in SHAPES] for _ in range(3))
    grads[1][100, 5] = request.param
    return w, grads, m


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("mu", [0.9, 0.0])
def test_the_orthogonalised_step_goes_on_along_its_momentum(g, bad, nesterov, mu):
    """M' = mu M, one fp32 product; W' = (1 - lr decay) W - lr O(U), U = mu M' (Nesterov) or M': as long a step as any, but
    without momentum, where U is 0 and weights decay."""
    w, grads, m = bad
    stats, _ = g.ar_grad_norm(grads, 1.0)
    plan = g.ar_ortho_plan(SHAPES)
    lr, decay, u = 0.125, 0.25, 2.0 ** -24
    new, momenta = [torch.empty_like(x) for x in w], [torch.empty_like(x) for x in m]
    g.ar_muon_step(plan, w, grads, m, lr, momentum=mu, weight_decay=decay, nesterov=nesterov, adjust="none",
                   params_out=new, momenta_out=momenta, clip=stats)
    assert all(torch.equal(a, b * mu) for a, b in zip(momenta, m))
    along = [torch.empty_like(x) for x in m]
    g.ar_orthogonalize(plan, [x * mu for x in momenta] if nesterov else momenta, outs=along)
    for a, b, o in zip(new, w, along):
        want = (1 - lr * decay) * b.double() - lr * o.double()
        # two products and a sum, of exact factors
        assert ((a.double() - want).abs() <= u * (2 * b.double().abs() + 2 * lr * o.double().abs())).all()
        # (the singular values of O are near 1, as many as the shorter side)
        length = (want - (1 - lr * decay) * b.double()).norm() / lr / min(b.shape) ** 0.5
        assert 0.6 < length < 1.3 if mu > 0 else length == 0


def test_adamw_skips_its_step_and_moves_on_zeros(g, bad):
    w, grads, m = bad
    v = [x.square() for x in m]
    stats, _, zeros = g.ar_grad_clip(grads, 1.0, outs=[torch.empty_like(x) for x in grads])
    assert all((x == 0).all() for x in zeros)
    keep = [[x.clone() for x in y] for y in (w, m, v)]
    g.ar_adamw_step(w, grads, m, v, 0.1, 5, clip=stats)
    for x, y in zip((w, m, v), keep):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    # the clipping call's zeros as gradients: moments decay, and the weights follow the first
    g.ar_adamw_step(w, zeros, m, v, 0.1, 5, betas=(0.5, 0.5))
    for a, b in zip(m + v, keep[1] + keep[2]):
        assert torch.equal(a, b * 0.5)
    for a, b, c in zip(w, keep[0], keep[1]):
        assert torch.equal(torch.sign(b - a), torch.sign(c))
