"""Microscaled blocks in float64: quantisation by search in the table of held values, and
the products as dense float64 products of the values held.

A block is 32 consecutive values of a row sharing one power of two 2^(e - 127);
e2m1 codes are 4-bit floats, int8 codes integers in units of 1/64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def n_blocks(cols: int) -> int:
    return -(-cols // BLOCK)


def quantize(x: np.ndarray, elem: str):
    """Codes (uint8 [rows][16 or 32 bytes per block]) and scale bytes ([rows][multiple of 16])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = n_blocks(cols)
    b = np.zeros((rows, nb, BLOCK))
    b.reshape(rows, nb * BLOCK)[:, :cols] = x
    finite = np.isfinite(b).all(axis=2)
    safe = np.where(finite[..., None], b, 0.0)
    top = np.abs(safe).max(axis=2)
    mant, ex = np.frexp(top)                       # top = mant · 2^ex, 0.5 <= mant < 1
    e = np.where(top > 0, ex - 1 - (2 if elem == "e2m1" else 0), -127)
    e = np.clip(e, -127, 127)
    v = np.ldexp(safe, -e[..., None])              # exact in float64
    if elem == "e2m1":
        d = np.abs(np.abs(v)[..., None] - E2M1)    # nearest held value, ties to the even code
        near = d == d.min(axis=-1, keepdims=True)
        even = near & (np.arange(8) % 2 == 0)
        code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1)).astype(np.uint8)
        code |= np.signbit(v).astype(np.uint8) << 3
        flat = code.reshape(rows, nb * BLOCK)
        codes = flat[:, 0::2] | (flat[:, 1::2] << 4)
    else:
        q = np.clip(np.rint(v * 64.0), -127, 127).astype(np.int8)
        codes = q.reshape(rows, nb * BLOCK).view(np.uint8)
    scales = np.zeros((rows, -(-nb // 16) * 16), np.uint8)
    scales[:, :nb] = np.where(finite, e + 127, 255).astype(np.uint8)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, cols: int, elem: str) -> np.ndarray:
    """The float64 values that the blocks stand for, [rows][cols]."""
    rows = codes.shape[0]
    nb = n_blocks(cols)
    if elem == "e2m1":
        flat = np.empty((rows, nb * BLOCK))
        for half in (0, 1):
            c = (codes.view(np.uint8) >> (4 * half)) & 15
            flat[:, half::2] = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    else:
        flat = codes.view(np.int8).astype(np.float64) / 64.0
    e = scales[:, :nb].astype(np.int64)
    s = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return (flat.reshape(rows, nb, BLOCK) * s[..., None]).reshape(rows, nb * BLOCK)[:, :cols]


def apply(D: np.ndarray, X: np.ndarray, add=None) -> np.ndarray:
    Y = np.einsum("tj,ij->ti", X, D)
    return Y if add is None else Y + add


def apply_t(D: np.ndarray, dY: np.ndarray, add=None) -> np.ndarray:
    dX = np.einsum("ti,ij->tj", dY, D)
    return dX if add is None else dX + add


def factor_grad(X, dY, U, V, add=None):
    """Gradients of L = <dY, X V Uᵀ> with respect to U, V and X (+ add)."""
    Z, G = X @ V, dY @ U
    dX = G @ V.T
    return dY.T @ Z, X.T @ G, dX if add is None else dX + add
