"""The norm, the block formats and the dense product in numpy fp64, from their
formulas: scales by their definition, codes by search for the nearest value.
Shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

from oracle.kv import E4M3, bf16, scale_of  # noqa: F401  (values of codes, of bf16 bits and of scale bytes)

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_rne(x):
    """fp64 to the nearest bf16, ties to even, as fp64 (finite values of bf16's normal range)."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(m * 256.0), e - 8)


def _codes(v, grid):
    """Index of the nearest of an increasing grid that starts at 0, ties to the even index; v >= 0."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantise(x, fmt):
    """Finite rows fp64 [rows][n] to (codes, scale bytes); "e2m1": 32 elements a scale, two codes a byte; "e4m3": 128."""
    grid, block, most, least = (E2M1, 32, 6.0, -126) if fmt == "e2m1" else (E4M3[:127], 128, 448.0, -127)
    rows, n = x.shape
    b = np.zeros((rows, -(-n // block) * block))
    b[:, :n] = x
    b = b.reshape(rows, -1, block)
    amax = np.abs(b).max(-1)
    k = np.zeros(amax.shape, np.int64)
    for i in np.ndindex(*amax.shape):
        if amax[i] > 0:
            while k[i] > least and amax[i] <= most * 2.0 ** (k[i] - 1):
                k[i] -= 1
            while k[i] < 127 and amax[i] > most * 2.0 ** k[i]:
                k[i] += 1
    q = _codes(np.minimum(np.abs(b) * 2.0 ** -k[..., None].astype(np.float64), most), grid)
    q = (q | np.where(np.signbit(b), len(E2M1) if fmt == "e2m1" else 128, 0)).reshape(rows, -1)[:, :n].astype(np.uint8)
    return (q[:, 0::2] | q[:, 1::2] << 4 if fmt == "e2m1" else q), (k + 127).astype(np.uint8)


def values(codes, scales, fmt):
    """What rows of codes and scale bytes stand for, fp64."""
    if fmt == "e2m1":
        q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
        v, block = np.concatenate([E2M1, -E2M1])[q], 32
    else:
        v, block = E4M3[codes], 128
    return v * np.repeat(scale_of(scales), block, -1)[:, :v.shape[1]]


def norm(r, weight, eps):
    """Rows fp64 (the residual added) over their root mean square, times weight."""
    with np.errstate(invalid="ignore"):
        r = r / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps)
    return r * (1.0 if weight is None else weight)


def linear(x, w):
    """(x w^T, sum of |x| |w|) of fp64 rows and weights."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def linear_tolerance(K, total):
    """Of a product in the tensor core's fp32 of K elements, `total` being the sum of their magnitudes: every step of 32
    elements, and every sum of split reductions, may lose 2^-22 of what the sums hold at most."""
    return (K / 32 + 10) * 2.0 ** -22 * total
