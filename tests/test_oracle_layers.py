"""Pins of the float64 oracles of the gated block, the norm and the loss over
the vocabulary (CPU only): gradients against central differences of the
forward functions, and facts of the definitions."""

import numpy as np
import pytest

from oracle import layers


def differences(f, x, h=1e-5):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradients_against_differences(kind):
    rng = np.random.default_rng(1)
    M, K, F, r, s = 4, 5, 6, 3, 0.7
    X, Wg, Wu, L1, L2, C = (rng.standard_normal(n) for n in ((M, K), (F, K), (F, K), (2, K, r), (2, r, F), (M, F)))
    loss = lambda X, L1, L2: float((layers.gated_fwd(X, Wg, Wu, L1, L2, s, kind)[0] * C).sum())  # noqa: E731
    dX, dL1, dL2, _, _ = layers.gated_bwd(X, Wg, Wu, L1, L2, s, kind, C)
    np.testing.assert_allclose(dX, differences(lambda x: loss(x, L1, L2), X), atol=1e-7)
    np.testing.assert_allclose(dL1, differences(lambda x: loss(X, x, L2), L1), atol=1e-7)
    np.testing.assert_allclose(dL2, differences(lambda x: loss(X, L1, x), L2), atol=1e-7)


def test_gelu_is_the_tanh_form():
    g = np.linspace(-6, 6, 101)
    a = layers.act(g, "gelu")[0]
    np.testing.assert_allclose(a, 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))), atol=1e-12)


@pytest.mark.parametrize("res", [False, True])
def test_norm_gradients_against_differences(res):
    rng = np.random.default_rng(2)
    M, K, eps = 3, 7, 1e-3
    x, r, w, C, Ch = (rng.standard_normal(n) for n in ((M, K), (M, K), (K,), (M, K), (M, K)))
    r = r if res else None

    def loss(x, w):
        y, h, _ = layers.norm_fwd(x, r, w, eps)
        return float((y * C).sum() + (h * Ch).sum())

    _, h, rstd = layers.norm_fwd(x, r, w, eps)
    dh, dw = layers.norm_bwd(C, h, rstd, w, Ch)
    np.testing.assert_allclose(dh, differences(lambda z: loss(z, w), x), atol=1e-7)
    np.testing.assert_allclose(dw, differences(lambda z: loss(x, z), w), atol=1e-7)


def test_head_gradients_against_differences():
    rng = np.random.default_rng(3)
    M, K, V = 6, 4, 5
    H, W = rng.standard_normal((M, K)), rng.standard_normal((V, K))
    labels = np.array([0, 4, -100, 2, 5, 2])         # rows 2 and 4 do not count
    weights = rng.random(M)
    for div in (0.0, 2.5):
        loss, nll, dH, dW, _, _ = layers.head_loss(H, W, labels, weights, div, 1.5)
        f = lambda H, W: 1.5 * layers.head_loss(H, W, labels, weights, div)[0]  # noqa: E731
        np.testing.assert_allclose(dH, differences(lambda z: f(z, W), H), atol=1e-8)
        np.testing.assert_allclose(dW, differences(lambda z: f(H, z), W), atol=1e-8)
        assert nll[2] == nll[4] == 0.0 and (dH[[2, 4]] == 0).all()
        assert abs(loss - float((weights * nll)[[0, 1, 3, 5]].sum() / (div or 4))) < 1e-12


def test_int8_values():
    codes, absmax = np.arange(-64, 64).astype(np.int8), np.array([127.0, 0.0], np.float32)
    v = layers.int8_values(codes, absmax)
    assert (v[:64] == codes[:64]).all() and (v[64:] == 0).all()
