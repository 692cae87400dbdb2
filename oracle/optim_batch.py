"""The optimiser step over many tensors (CPU oracle). Test infrastructure only.

Norm and update are those of oracle/optim.py over the concatenated tensors
(float64). The 8-bit state of one vector, per block of 256 values x of a
tensor (the last block may be short): top = max|x|; scale = top / 448; the
stored value is the E4M3 value nearest to x 448 / top, times scale; a top
below 2^-100 stores zeros. The second moment is stored as its square root,
where a value above 0 is stored as at least 2^-9 (the smallest E4M3 step).

``encode`` works in the dtype of its input, one rounding per operation: in
float32 it gives the codes bit for bit, in float64 the definition.
"""

from __future__ import annotations

import numpy as np

from oracle import nf4, optim

BLOCK = 256
STEP = 2.0 ** -9


def span(n: int) -> int:
    """Elements that a tensor of n values takes in a state array."""
    return -(-n // BLOCK) * BLOCK


def offsets(numel) -> list[int]:
    at = [0]
    for n in numel:
        at.append(at[-1] + span(n))
    return at


def encode(x: np.ndarray, keep: bool):
    """(codes uint8 [span], scale [blocks]) of one tensor's values; padding gets code 0."""
    t = x.dtype.type
    b = np.zeros(span(x.size), x.dtype)
    b[:x.size] = x
    b = b.reshape(-1, BLOCK)
    top = np.abs(b).max(axis=1) if b.size else np.zeros(0, x.dtype)
    top = np.where(top < t(2.0 ** -100), t(0), top)
    with np.errstate(divide="ignore"):
        inv = np.where(top > 0, t(448) / top, t(0)).astype(x.dtype)
    y = (b * inv[:, None]).astype(x.dtype)
    if keep:
        y = np.where(y > 0, np.maximum(y, t(STEP)), y)
    return nf4.e4m3_encode(y.astype(np.float32)).reshape(-1), (top / t(448)).astype(x.dtype)


def decode(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The fp32 values of a state array: RN32(value(code) scale)."""
    v = nf4.e4m3_decode(codes).astype(np.float32).reshape(-1, BLOCK)
    return (v * scale.astype(np.float32)[:, None]).reshape(-1)


def clip(grads, max_norm: float):
    """(coef, norm) over all tensors, in float64."""
    flat = np.concatenate([np.asarray(g, np.float64).reshape(-1) for g in grads]) if len(grads) else np.zeros(0)
    return optim.clip_coef(flat, max_norm), optim.grad_norm(flat)
