"""The rest of a training step (CPU oracle, float64). Test infrastructure only.

The gated feed-forward block's first half with adapters, the root-mean-square
norm with the residual's addition, softmax cross entropy of hidden states
against a head's weight, and the values that 8 bits hold, straight from their
definitions. Inputs are bf16 bit patterns (uint16, widened exactly) or floats.
"""

from __future__ import annotations

import numpy as np

from .linear import linear_bwd, linear_fwd, widen

BLOCK = 64


def int8_values(codes, absmax):
    """code * RN32(absmax / 127), flat, in float64."""
    scale = (np.asarray(absmax, np.float32) / np.float32(127.0)).astype(np.float64)
    return (codes.astype(np.float64).reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def act(g, kind: str):
    """act(g), act'(g) and z of act(g) = g sigmoid(z)."""
    if kind == "silu":
        z, dz = g, np.ones_like(g)
    else:
        c = np.sqrt(8.0 / np.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 3.0 * 0.044715 * g ** 2)
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-z))
    return g * p, p + g * p * (1.0 - p) * dz, z


def gate_up(X, Wg, Wu, L1, L2, s):
    G, Tg = linear_fwd(X, Wg, L1[0], L2[0], s)
    U, Tu = linear_fwd(X, Wu, L1[1], L2[1], s)
    return G, U, np.stack([Tg, Tu])


def gated_fwd(X, Wg, Wu, L1, L2, s, kind):
    """(A, G, U, T)."""
    G, U, T = gate_up(X, Wg, Wu, L1, L2, s)
    return act(G, kind)[0] * U, G, U, T


def gated_bwd(X, Wg, Wu, L1, L2, s, kind, dA, GU=None):
    """(dX, dL1, dL2, dG, dU); GU: kept (G, U) in their place."""
    G, U = gate_up(X, Wg, Wu, L1, L2, s)[:2] if GU is None else GU
    a, d, _ = act(G, kind)
    dA = widen(dA)
    dG, dU = dA * U * d, dA * a
    xg, g1, g2 = linear_bwd(X, Wg, L1[0], L2[0], s, dG)
    xu, u1, u2 = linear_bwd(X, Wu, L1[1], L2[1], s, dU)
    return xg + xu, np.stack([g1, u1]), np.stack([g2, u2]), dG, dU


def norm_fwd(x, res, w, eps):
    """(y, h, rstd)."""
    h = widen(x) + (0.0 if res is None else widen(res))
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * (1.0 if w is None else widen(w)), h, rstd


def norm_bwd(dy, h, rstd, w, dres):
    """(dh, dweight) for the given rstd."""
    dy, h, r = widen(dy), widen(h), widen(rstd)[:, None]
    xh = h * r
    wd = dy * (1.0 if w is None else widen(w))
    dh = r * (wd - xh * (wd * xh).mean(axis=1, keepdims=True))
    return dh + (0.0 if dres is None else widen(dres)), (dy * xh).sum(axis=0)


def head_loss(H, W, labels, weights=None, divisor=0.0, scale=1.0):
    """(loss, nll, dH, dW, softmax, g): g the factor of each row's gradient."""
    H, W = widen(H), widen(W)
    V = W.shape[0]
    on = (labels >= 0) & (labels < V)
    at = np.where(on, labels, 0)
    S = H @ W.T
    with np.errstate(invalid="ignore", over="ignore"):
        top = S.max(axis=1, keepdims=True) if len(S) else S[:, :1]
        e = np.exp(S - top)
        total = e.sum(axis=1, keepdims=True)
        p = e / total
        lse = (np.log(total) + top)[:, 0]
    nll = np.where(on, lse - np.take_along_axis(S, at[:, None], 1)[:, 0], 0.0)
    w = np.where(on, 1.0 if weights is None else np.asarray(weights, np.float64), 0.0)
    w = w / (float(divisor) if divisor else max(int(on.sum()), 1))
    g = scale * w
    D = p.copy()
    np.put_along_axis(D, at[:, None], np.take_along_axis(D, at[:, None], 1) - 1.0, 1)
    D = np.where(on[:, None], g[:, None] * D, 0.0)
    loss = float((w * np.where(on, nll, 0.0)).sum())
    return loss, nll, D @ W, D.T @ np.where(on[:, None], H, 0.0), p, g
