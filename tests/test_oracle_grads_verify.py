"""The 64-bit references of the gradient norm, AdamW and the verification of drafted tokens, against
worked numbers, torch and their own laws."""

import numpy as np
import pytest
import torch

from oracle import grads, verify


def test_norm_of_worked_numbers():
    stats, norms = grads.norm([np.array([3.0]), np.array([[0.0, 4.0]]), np.zeros(0)], max_norm=1.0, eps=0.0)
    assert stats.tolist() == [5.0, 0.2, 1.0, 1.0] and norms.tolist() == [3.0, 4.0, 0.0]
    stats, norms = grads.norm([np.array([3.0, -8.0]), np.array([4.0])], max_norm=1.0, eps=0.0, kind="max", grad_scale=0.5)
    assert stats.tolist() == [4.0, 0.25, 1.0, 1.0] and norms.tolist() == [4.0, 2.0]
    assert grads.norm([np.array([np.nan, 1.0])])[0][1:].tolist() == [0.0, 1.0, 0.0]
    _, _, (out,) = grads.clip([np.array([30.0, 40.0])], 5.0, eps=0.0)
    assert np.allclose(out, [3.0, 4.0], rtol=1e-15)


@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_adamw_is_torchs(decay):
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(50, generator=gen, dtype=torch.float64)
    leaf = w.clone().requires_grad_()
    opt = torch.optim.AdamW([leaf], lr=0.01, betas=(0.9, 0.95), eps=1e-6, weight_decay=decay)
    x, m, v = w.numpy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        leaf.grad = torch.randn(50, generator=gen, dtype=torch.float64)
        opt.step()
        x, m, v = grads.adamw(x, leaf.grad.numpy() * 2, m, v, t, 0.01, (0.9, 0.95), 1e-6, decay, scale=0.5)
        # the same few operations in another order, in 64 bits: at most some 2^-50 a step
        assert np.allclose(x, leaf.detach().numpy(), rtol=1e-13, atol=1e-14)


@pytest.mark.parametrize("seed", range(4))
def test_emitted_tokens_have_the_targets_distribution(seed):
    rng = np.random.default_rng(seed)
    p, q = (verify.softmax(rng.normal(size=40) * 2) for _ in range(2))
    assert np.allclose(verify.emitted(p, q), p, rtol=1e-12, atol=1e-15)
    one = np.zeros(40)
    one[7] = 1.0
    assert np.allclose(verify.emitted(p, one), p, rtol=1e-12, atol=1e-15)


def test_verify_worked_example():
    # p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4): the draft 1 stands below 1/2, else token 0 is drawn
    p, q = np.log([[0.5, 0.25, 0.25]] * 2), np.log([[0.25, 0.5, 0.25]])
    for u, v, tokens, a in ((0.4, 0.6, [1, 1], 1), (0.6, 0.9, [0, -1], 0), (0.4, 0.9, [1, 2], 1)):
        got = verify.verify(p, [1], np.array([u, v]), [0, 1], q)
        assert got[1].tolist() == tokens and got[0].tolist() == [a]
    # without a distribution: 1 stands below 1/4; behind it, (1/2, 0, 1/4) is drawn from
    assert verify.verify(p, [1], np.array([0.3, 0.7]), [0, 1])[1].tolist() == [2, -1]
    # two sequences, one without drafts; greedy takes the first of equals
    got = verify.verify(np.log([[0.5, 0.5], [0.2, 0.8], [0.2, 0.8]]), [1], None, [0, 0, 1], greedy=True)
    assert got[1].tolist() == [0, 1, 1] and got[0].tolist() == [0, 1]
    assert np.isnan(verify.verify(np.array([[np.nan, 0.0]]), [], np.array([0.5]), [0, 0])[2][0])
