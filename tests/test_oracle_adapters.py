"""Pins of the float64 oracles behind the many-adapter operators (CPU only):
their gradients against central differences of their forward functions, and
the 8-bit optimiser state's format facts."""

import numpy as np
import pytest

from oracle import linear, multi, nf4, optim_batch, preference


def differences(f, x, h):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_multi_gradients_against_differences():
    rng = np.random.default_rng(1)
    M, K, N, r, A = 7, 5, 4, 3, 3
    ids = np.array([0, 2, -1, 0, 3, 2, 2])       # adapter 1 has no rows, ids -1 and 3 are none
    X, W, L1, L2 = (rng.standard_normal(s) for s in ((M, K), (N, K), (A, K, r), (A, r, N)))
    s, C = np.array([0.5, 1.0, 2.0]), rng.standard_normal((M, N))
    dX, dL1, dL2 = multi.multi_bwd(X, W, ids, L1, L2, s, C)
    loss = lambda X, L1, L2: float((multi.multi_fwd(X, W, ids, L1, L2, s)[0] * C).sum())  # noqa: E731
    # the loss is at most quadratic in each argument: differences have no truncation error
    np.testing.assert_allclose(dX, differences(lambda x: loss(x, L1, L2), X, 1e-3), atol=1e-9)
    np.testing.assert_allclose(dL1, differences(lambda x: loss(X, x, L2), L1, 1e-3), atol=1e-9)
    np.testing.assert_allclose(dL2, differences(lambda x: loss(X, L1, x), L2, 1e-3), atol=1e-9)
    assert (dL1[1] == 0).all() and (dL2[1] == 0).all()


def test_multi_of_one_adapter_is_the_linear():
    rng = np.random.default_rng(2)
    X, W, L1, L2, dY = (rng.standard_normal(s) for s in ((6, 5), (4, 5), (1, 5, 2), (1, 2, 4), (6, 4)))
    Y, T = multi.multi_fwd(X, W, np.zeros(6, int), L1, L2, [0.25])
    Yr, Tr = linear.linear_fwd(X, W, L1[0], L2[0], 0.25)
    np.testing.assert_array_equal(T, Tr)
    np.testing.assert_allclose(Y, Yr, rtol=1e-14)
    for got, ref in zip(multi.multi_bwd(X, W, np.zeros(6, int), L1, L2, [0.25], dY),
                        linear.linear_bwd(X, W, L1[0], L2[0], 0.25, dY)):
        np.testing.assert_allclose(got.reshape(ref.shape), ref, rtol=1e-14)


@pytest.mark.parametrize("eps", [0.0, 0.3])
def test_preference_gradient_against_differences(eps):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 3, 5))
    labels = rng.integers(0, 5, (4, 3))
    labels[1, 0] = -100
    labels[2, 2] = 5
    ref = rng.standard_normal((4, 3))
    loss, rewards, lp, grad, w, _ = preference.preference(x, labels, ref, 0.7, eps, 1.5)
    num = differences(lambda z: 1.5 * preference.preference(z, labels, ref, 0.7, eps)[0], x, 1e-5)
    np.testing.assert_allclose(grad, num, atol=1e-9)
    assert (lp[1, 0], lp[2, 2]) == (0.0, 0.0) and (grad[1, 0] == 0).all() and (grad[2, 2] == 0).all()


def test_preference_at_the_reference():
    """A policy equal to its reference: loss log 2, weights beta / (2 P)."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 4, 6))
    labels = rng.integers(0, 6, (2, 4))
    lp = preference.preference(x, labels, np.zeros((2, 4)), 0.1, 0.0)[2]
    loss, rewards, _, _, w, _ = preference.preference(x, labels, lp, 0.1, 0.0)
    assert loss == pytest.approx(np.log(2), rel=1e-15) and (rewards == 0).all()
    np.testing.assert_allclose(w, [-0.05, 0.05], rtol=1e-15)


def test_state_codes():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal(1000) * np.exp(3 * rng.standard_normal(1000))).astype(np.float32)
    codes, scale = optim_batch.encode(x, False)
    assert codes.shape == (1024,) and scale.shape == (4,) and (codes[1000:] == 0).all()
    back = optim_batch.decode(codes, scale)[:1000]
    top = np.repeat(scale, 256)[:1000]
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * top) * (1 + 1e-6)).all()
    for b in range(4):                                   # the block's largest value keeps the largest code
        k = np.abs(x[256 * b:256 * b + 256]).argmax() + 256 * b
        assert abs(nf4.e4m3_decode(codes)[k]) == 448.0
    codes, scale = optim_batch.encode(np.abs(x), True)
    assert (optim_batch.decode(codes, scale)[:1000][x != 0] > 0).all()
    assert optim_batch.offsets([1, 0, 256, 257]) == [0, 256, 256, 512, 1024]
