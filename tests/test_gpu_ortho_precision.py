"""SPLIT, the default of fp32 results, against elementary fp32 operations: errors against 64 bits at most half as large
again, for the mean over a few inputs. Matrices of a few hundred rows, and fewer, are where fp32 operations round least."""

import pytest
import torch

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module")
def g():
    from gradient_sync_gb300 import build

    build.build()
    import gradient_sync_gb300 as g

    return g


def steps(u, dtype):
    x = u.to(dtype)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        a = x @ x.T
        x = A * x + (B * a + C * (a @ a)) @ x
    return x.T if u.shape[0] > u.shape[1] else x


@pytest.mark.parametrize("shape", [(77, 2049), (130, 4000), (300, 3000), (3000, 100), (1000, 333), (512, 2048),
                                   (200, 200), (1024, 4096)])
def test_as_precise_as_fp32_operations(g, shape):
    r, c = shape
    errors = {"own": 0.0, "fp32": 0.0}
    for seed in range(5):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        k = min(r, c, 16)  # a few strong directions over noise
        u = torch.randn(r, k, generator=gen, device="cuda") * torch.linspace(1, 0.2, k, device="cuda")
        m = u @ torch.randn(k, c, generator=gen, device="cuda") * 0.5 + torch.randn(r, c, generator=gen, device="cuda")
        want = steps(m, torch.float64)
        own = g.ar_orthogonalize(g.ar_ortho_plan([shape]), [m])[0]
        for name, x in (("own", own), ("fp32", steps(m, torch.float32))):
            errors[name] += float((x.double() - want).norm() / want.norm())
    assert errors["own"] <= 1.5 * errors["fp32"], errors
