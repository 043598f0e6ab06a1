"""The orthogonalised update's oracle on the CPU: the products against the singular values."""

import numpy as np
import pytest

from oracle import ortho


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (9, 1), (5, 5), (7, 30), (30, 7)])
def test_products_act_on_the_singular_values(shape):
    u = np.random.default_rng(0).normal(size=shape)
    np.testing.assert_allclose(ortho.newton_schulz(u), ortho.newton_schulz_svd(u), atol=1e-12)


def test_singular_values_end_near_one():
    u = np.random.default_rng(1).normal(size=(40, 60))
    s = np.linalg.svd(ortho.newton_schulz(u), compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.2


def test_transpose_scale_and_zero():
    u = np.random.default_rng(2).normal(size=(8, 20))
    np.testing.assert_allclose(ortho.newton_schulz(u.T), ortho.newton_schulz(u).T, atol=1e-13)
    np.testing.assert_allclose(ortho.newton_schulz(1e6 * u), ortho.newton_schulz(u), atol=1e-6)
    assert not ortho.newton_schulz(0 * u).any()


def test_step_by_hand():
    # one entry: the orthogonal matrix of a 1 x 1 update is the polynomial of +-1, five times
    s = 1.0
    for _ in range(5):
        s = 3.4445 * s - 4.775 * s**3 + 2.0315 * s**5
    w, m = ortho.muon_step([[2.0]], [[4.0]], [[1.0]], lr=0.1, momentum=0.5, weight_decay=0.2, grad_scale=0.25, eps=0.0)
    assert np.allclose(m, 1.5) and np.allclose(w, 2.0 * 0.98 - 0.1 * s)
