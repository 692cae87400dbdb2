"""The preference loss (CPU oracle, float64). Test infrastructure only.

A policy's paired log ratios against a reference (Rafailov et al., "Direct
Preference Optimization", NeurIPS 2023, eq. 7), with label smoothing e:

    lp[s][t]  = x[y] - log sum_v exp(x[v]),  x = logits[s][t], y = labels[s][t]
    reward[s] = beta sum_t (lp - ref)       over the positions with 0 <= y < V
    h_p       = reward[p] - reward[P + p]
    loss      = mean_p (1 - e) softplus(-h_p) + e softplus(h_p)

and, by d softplus(-h)/dh = -sigmoid(-h), d softplus(h)/dh = sigmoid(h) = 1 - sigmoid(-h),

    d loss / d lp[p] = (beta / P) (e - sigmoid(-h_p)),  the opposite for P + p,
    d lp / d x       = onehot(y) - softmax(x).
"""

from __future__ import annotations

import numpy as np


def softplus(z):
    return np.maximum(z, 0.0) + np.log1p(np.exp(-np.abs(z)))


def preference(logits, labels, ref, beta: float, eps: float, scale: float = 1.0):
    """(loss, rewards [S], lp [S][T], dlogits, weight [S], softmax) in float64."""
    x = np.asarray(logits, np.float64)
    S, T, V = x.shape
    P = S // 2
    on = (labels >= 0) & (labels < V)
    y = np.where(on, labels, 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = x.max(axis=2, keepdims=True) if T else np.zeros((S, 0, 1))
        e = np.exp(x - top)
        total = e.sum(axis=2, keepdims=True)
        lse = (top + np.log(total))[..., 0]
        lp = np.where(on, np.take_along_axis(x, y[..., None], 2)[..., 0] - lse, 0.0)
        q = e / total
    d = np.where(on, lp - np.where(on, ref, 0.0).astype(np.float64), 0.0)
    rewards = beta * d.sum(axis=1)
    h = rewards[:P] - rewards[P:]
    loss = float(np.mean((1.0 - eps) * softplus(-h) + eps * softplus(h))) if P else 0.0
    w = (scale * beta / max(P, 1)) * (eps - 1.0 / (1.0 + np.exp(h)))
    w = np.concatenate([w, -w])
    grad = -q.copy()
    np.put_along_axis(grad, y[..., None], np.take_along_axis(grad, y[..., None], 2) + 1.0, 2)
    grad = np.where(on[..., None], w[:, None, None] * grad, 0.0)
    return loss, rewards, lp, grad, w, q
