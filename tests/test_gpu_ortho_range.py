"""The orthogonalised update of matrices of any size of element, on a GB300 against its oracle in 64 bits.

The tolerance is test_gpu_ortho.py's for SPLIT, 3e-5 relative to the norm sqrt(m) of an orthogonal m x n matrix: a
norm that is summed at another power of two is rounded like one that is not."""

import numpy as np
import pytest
import torch

from oracle import ortho

pytestmark = pytest.mark.gpu

SPLIT = 3e-5
SHAPES = [(96, 200), (201, 96), (130, 133), (1, 77)]  # wide, tall, read an element at a time, one row


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def noise(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def check(got, m, eps):
    want = ortho.newton_schulz(m.double().cpu().numpy(), eps=eps)
    err = np.linalg.norm(got.double().cpu().numpy() - want)
    assert err <= SPLIT * min(m.shape) ** 0.5, (err, tuple(m.shape))


@pytest.mark.parametrize("power", [-138, -110, -80, -41, -40, -39, 39, 40, 41, 80, 110, 124])
def test_powers_of_two(g, power):
    """At eps = 0 the result does not depend on the input's scale, over all of fp32's range."""
    mats = [noise(s, i) * 2.0 ** power for i, s in enumerate(SHAPES)]
    plan = g.ar_ortho_plan(SHAPES, eps=0.0)
    for m, o in zip(mats, g.ar_orthogonalize(plan, mats)):
        assert torch.isfinite(m).all() and m.any()
        check(o, m, 0.0)


def test_power_of_two_bits(g):
    mats = [noise(s, i) for i, s in enumerate(SHAPES)]
    plan = g.ar_ortho_plan(SHAPES, eps=0.0)
    want = g.ar_orthogonalize(plan, mats)
    for power in (-110, 110):
        got = g.ar_orthogonalize(plan, [m * 2.0 ** power for m in mats])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("span", [(-120, 120), (-60, 60), (-140, -30), (30, 126)])
def test_elements_far_apart(g, span):
    """Rows, and single elements, whose sizes lie up to 240 powers of two apart."""
    mats = []
    for i, s in enumerate(SHAPES):
        rows = torch.linspace(*span, s[0], device="cuda")[:, None].expand(s)
        cols = torch.linspace(*span, s[1], device="cuda")[None, :].expand(s)
        mats.append(noise(s, i).clamp(-3, 3) * torch.exp2((rows if i % 2 else cols).double()).float())
    plan = g.ar_ortho_plan(SHAPES, eps=0.0)
    for m, o in zip(mats, g.ar_orthogonalize(plan, mats)):
        assert torch.isfinite(m).all()
        check(o, m, 0.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e25, 1e38, 1e-25])
def test_default_eps_and_steps(g, scale, dtype):
    """The optimiser's step on gradients of any size, and the update's eps where it is all that counts."""
    kind = "bf16" if dtype == torch.bfloat16 else "f32"
    grads = [(noise(s, i).clamp(-3, 3) * scale).to(dtype) for i, s in enumerate(SHAPES)]
    plan = g.ar_ortho_plan(SHAPES, kind, "f32")
    for m, o in zip(grads, g.ar_orthogonalize(plan, grads)):
        check(o, m, np.float32(1e-7))
    params, momenta = [torch.zeros(s, device="cuda") for s in SHAPES], [torch.zeros(s, device="cuda") for s in SHAPES]
    g.ar_muon_step(plan, params, grads, momenta, lr=1.0, momentum=0.5, nesterov=False, adjust="none")
    for p, m, q in zip(params, grads, momenta):
        assert torch.equal(q, m.float())
        check(-p, m, np.float32(1e-7))


@pytest.mark.parametrize("power", [-100, -50, 0, 50, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(g, bad, power):
    mats = [noise(s, i) * 2.0 ** power for i, s in enumerate(SHAPES)]
    for m in mats:
        m[0, m.shape[1] // 2] = bad
    mats.append(torch.zeros(7, 9, device="cuda"))
    out = g.ar_orthogonalize(g.ar_ortho_plan([*SHAPES, (7, 9)]), mats)
    assert all(torch.isnan(o).all() for o in out[:-1]) and not out[-1].any()
