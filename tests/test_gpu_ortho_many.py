"""Plans of more matrices than run together (64), as the optimiser step of a whole model has, on a GB300 against the
oracle in 64 bits.

Tolerances are those of test_gpu_ortho.py: 6e-3 (HALF) and 3e-5 (SPLIT) of sqrt(m). HALF's takes it that the errors
of early steps are not amplified, which holds in the mean over many singular values and not for each: the steps'
polynomial p has slopes up to 3.4. So matrices of fewer than 8 rows have what one step's rounding, 1.5e-3 of sqrt(m)
spread evenly over the elements, becomes in the steps behind it: to first order a component between the i-th left and
the j-th right singular vector is carried on by (p(s_i) - p(s_j)) / (s_i - s_j) and (p(s_i) + p(s_j)) / (s_i + s_j),
and one outside the right vectors by p(s_i) / s_i. Three times that, since a few elements do not average.
"""

import numpy as np
import pytest
import torch

from oracle import ortho

pytestmark = pytest.mark.gpu

TOL = {"half": 6e-3, "split": 3e-5}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def shapes_of(n):
    """Sizes from 1 to 600, so that every group of 64 has tall, wide, square and thin ones."""
    rng = np.random.default_rng(n)
    out = [(int(np.exp(rng.uniform(0, np.log(600)))), int(np.exp(rng.uniform(0, np.log(600))))) for _ in range(n)]
    out[-1], out[n // 2], out[0] = (130, 5), (5, 130), (64, 64)
    return out


def host(t):
    return t.double().cpu().numpy()


def carried(u):
    """Frobenius norm of the steps' rounding errors in HALF, to first order (see above)."""
    m, n = min(u.shape), max(u.shape)
    s = np.linalg.svd(u / np.linalg.norm(u), compute_uv=False)
    a, b, c = ortho.COEFFICIENTS
    inside, outside = np.zeros((m, m)), np.zeros(m)
    for _ in range(5):
        x, y = s[:, None], s[None, :]
        # divided differences of p(x) = a x + b x^3 + c x^5 at x and y, and at x and -y
        apart = a + b * (x * x + x * y + y * y) + c * (x**4 + x**3 * y + x * x * y * y + x * y**3 + y**4)
        joined = a + b * (x * x - x * y + y * y) + c * (x**4 - x**3 * y + x * x * y * y - x * y**3 + y**4)
        inside = inside * np.maximum(np.abs(apart), np.abs(joined)) + 1.5e-3 / n ** 0.5
        outside = outside * np.abs(a + b * s * s + c * s**4) + 1.5e-3 / n ** 0.5
        s = np.abs(a * s + b * s**3 + c * s**5)
    return np.sqrt((inside ** 2).sum() + (n - m) * (outside ** 2).sum())


def check(got, want, tol, rounded, u=None):
    over = np.maximum(np.abs(host(got) - want) - rounded * np.abs(want), 0)
    bound = tol * min(want.shape) ** 0.5
    if u is not None and min(u.shape) < 8:
        bound = max(bound, 3 * carried(u))
    assert np.sqrt((over ** 2).sum()) <= bound, (want.shape, np.sqrt((over ** 2).sum()), bound)


@pytest.mark.parametrize("precision,src,dst", [("half", "bf16", "bf16"), ("split", "f32", "f32")])
@pytest.mark.parametrize("n", [64, 65, 112, 129, 192])
def test_many_matrices(g, n, precision, src, dst):
    shapes = shapes_of(n)
    rng = np.random.default_rng(1)
    mats = [torch.tensor(rng.normal(size=s), dtype=TYPES[src], device="cuda") for s in shapes]
    plan = g.ar_ortho_plan(shapes, src, dst, precision=precision)
    outs = g.ar_orthogonalize(plan, mats)
    for m, o in zip(mats, outs):
        u = host(m)
        check(o, ortho.newton_schulz(u), TOL[precision], 2.0 ** -8 if dst == "bf16" else 0.0,
              u if precision == "half" else None)
    # with the same workspace, call after call, and in place
    room = torch.empty(g.ar_ortho_workspace(plan), dtype=torch.uint8, device="cuda").fill_(255)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(g.ar_orthogonalize(plan, mats, workspace=room), outs))
    g.ar_orthogonalize(plan, mats, outs=mats, workspace=room)
    assert all(torch.equal(a, b) for a, b in zip(mats, outs))
    assert g.ar_device_status() == g.AR_OK


@pytest.mark.parametrize("src,dst", [("f32", "bf16"), ("f32", "f32")])
def test_step_of_a_model_of_16_layers(g, src, dst):
    """Seven projections a layer, four square, three of them wide or tall: 112 matrices."""
    shapes = [s for _ in range(16) for s in [(96, 96)] * 4 + [(96, 384)] * 2 + [(384, 96)]]
    rng = np.random.default_rng(2)
    grads = [torch.tensor(rng.normal(size=s) * 1e-3, dtype=TYPES[src], device="cuda") for s in shapes]
    params = [torch.tensor(rng.normal(size=s) * 0.02, dtype=TYPES[dst], device="cuda") for s in shapes]
    momenta = [torch.tensor(rng.normal(size=s) * 2e-3, dtype=torch.float32, device="cuda") for s in shapes]
    kw = dict(lr=0.02, momentum=0.9, weight_decay=0.1, nesterov=True, adjust="shape", grad_scale=0.5)
    want = [ortho.muon_step(host(p), host(q), host(m), **kw) for p, q, m in zip(params, grads, momenta)]
    g.ar_muon_step(g.ar_ortho_plan(shapes, src, dst), params, grads, momenta, **kw)
    tol = TOL["half" if dst == "bf16" else "split"]
    for s, p, m, (w, m64) in zip(shapes, params, momenta, want):
        assert np.abs(host(m) - m64).max() <= 2.0 ** -22 * np.abs(m64).max()
        check(p, w, tol * 0.02 * ortho.adjust_factor(*s, "shape"), 2.0 ** -8 if dst == "bf16" else 2.0 ** -22)
