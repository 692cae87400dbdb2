"""The QLoRA linear with an adapter per row (CPU oracle, float64). Test infrastructure only.

Every row goes through oracle/linear.py's layer with its own adapter; a row
whose id lies outside [0, A) has none:

    Y[m]   = X[m] W^T + s_a (X[m] L1_a) L2_a
    dX[m]  = dY[m] W + s_a (dY[m] L2_a^T) L1_a^T
    dL1_a  = s_a sum_{m of a} X[m]^T (dY[m] L2_a^T)
    dL2_a  = s_a sum_{m of a} (X[m] L1_a)^T dY[m]
"""

from __future__ import annotations

import numpy as np

from oracle.linear import linear_bwd, widen


def rows_of(ids, A: int):
    """The rows of each adapter, in order."""
    ids = np.asarray(ids)
    return [np.nonzero(ids == a)[0] for a in range(A)]


def multi_fwd(X, Wt, ids, L1, L2, scale):
    """(Y, T) in float64; T is zero for rows without an adapter."""
    X, Wt, L1, L2 = widen(X), widen(Wt), widen(L1), widen(L2)
    Y = X @ Wt.T
    T = np.zeros((X.shape[0], L1.shape[2]))
    for a, at in enumerate(rows_of(ids, L1.shape[0])):
        T[at] = X[at] @ L1[a]
        Y[at] += float(scale[a]) * (T[at] @ L2[a])
    return Y, T


def multi_bwd(X, Wt, ids, L1, L2, scale, dY):
    """(dX, dL1, dL2) in float64."""
    X, Wt, L1, L2, dY = widen(X), widen(Wt), widen(L1), widen(L2), widen(dY)
    dX = dY @ Wt
    dL1, dL2 = np.zeros(L1.shape), np.zeros(L2.shape)
    for a, at in enumerate(rows_of(ids, L1.shape[0])):
        if len(at):
            dX[at], dL1[a], dL2[a] = linear_bwd(X[at], Wt, L1[a], L2[a], float(scale[a]), dY[at])
    return dX, dL1, dL2
