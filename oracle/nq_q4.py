"""fp64 oracle of the linears with 4-bit weights and group scales.

    W[i, j] = s[i, j // G] (q[i, j] - z[i, j // G])      y = x W^T

q: codes in 0..15 (m x n); s, z: m x ceil(n / G) (z None: 8 everywhere).
"""
from __future__ import annotations

import numpy as np


def weight(q, s, z, G: int) -> np.ndarray:
    """The dense weight, element by element from the definition."""
    q = np.asarray(q, np.float64)
    s = np.asarray(s, np.float64)
    z = np.full(s.shape, 8.0) if z is None else np.asarray(z, np.float64)
    g = np.arange(q.shape[1]) // G
    return s[:, g] * (q - z[:, g])


def linear(x, q, s, z, G: int) -> np.ndarray:
    return np.asarray(x, np.float64) @ weight(q, s, z, G).T


def magnitude(x, q, s, z, G: int) -> np.ndarray:
    """sum_j |W[i, j] x[b, j]|: what the rounding of a sum is measured against."""
    return np.abs(np.asarray(x, np.float64)) @ np.abs(weight(q, s, z, G)).T
