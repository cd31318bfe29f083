"""The norm's oracle against torch's autograd on an independent formula, central
differences and closed forms."""
import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("T,d", [(1, 8), (5, 24), (3, 256)])
def test_forward_and_gradients_against_autograd(T, d):
    g = torch.Generator().manual_seed(T + d)
    x, res, dy, ds = (torch.randn(T, d, generator=g, dtype=torch.float64) for _ in range(4))
    gamma = torch.randn(d, generator=g, dtype=torch.float64)
    for t in (x, res, gamma):
        t.requires_grad_()
    s = x + res
    y = s / (s.pow(2).sum(1, keepdim=True) / d + 1e-5).pow(0.5) * gamma
    got, rstd = oracle.rms_norm(s.detach().numpy(), gamma.detach().numpy(), 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-13, atol=1e-13)
    ((y * dy).sum() + (s * ds).sum()).backward()
    dx, dg = oracle.rms_norm_bwd(dy.numpy(), s.detach().numpy(), rstd, gamma.detach().numpy(), ds.numpy())
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dx, res.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dg, gamma.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    s, dy, gamma = rng.standard_normal((2, 16)), rng.standard_normal((2, 16)), rng.standard_normal(16)

    def loss(s_, g_):
        return float((oracle.rms_norm(s_, g_, 1e-6)[0] * dy).sum())
    dx, dg = oracle.rms_norm_bwd(dy, s, oracle.rms_norm(s, gamma, 1e-6)[1], gamma)
    h = 1e-5
    for i in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[i] = h
        assert abs((loss(s + e, gamma) - loss(s - e, gamma)) / (2 * h) - dx[i]) < 1e-8
    for i in range(16):
        e = np.zeros(16)
        e[i] = h
        assert abs((loss(s, gamma + e) - loss(s, gamma - e)) / (2 * h) - dg[i]) < 1e-8


def test_closed_forms():
    y, r = oracle.rms_norm(np.full((1, 4), 3.0), np.ones(4), 0.0)
    assert np.array_equal(y, np.ones((1, 4))) and r[0] == 1 / 3
    y, r = oracle.rms_norm(np.zeros((1, 4)), np.ones(4), 0.25)
    assert np.array_equal(y, np.zeros((1, 4))) and r[0] == 2.0
    # the norm does not change with the row's size: the gradient along the row is zero
    s = np.array([[1.0, -2.0, 3.0, 0.5]])
    dx, _ = oracle.rms_norm_bwd(np.array([[1.0, 4.0, -1.0, 2.0]]), s, oracle.rms_norm(s, np.ones(4), 0.0)[1],
                                np.ones(4))
    assert abs((dx * s).sum()) < 1e-14
