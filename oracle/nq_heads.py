"""fp64 oracle of the norms and the rotation of heads and of their gradients.

    n = x r w,  r = (mean x^2 + eps)^-1/2    (y_a, y_b) = (n_a cos p - n_b sin p, n_a sin p + n_b cos p)

x (tokens, heads, D); w the weight plus its offset, or None for 1; angles (tokens, R / 2).
"""
from __future__ import annotations

import numpy as np


def angles(positions, inv_freq, sections) -> np.ndarray:
    """positions (axes, tokens) x inv_freq (R / 2) -> (tokens, R / 2), less whole turns;
    the product and its remainder in extended precision."""
    f = np.asarray(inv_freq, np.float64).astype(np.longdouble)
    p = np.asarray(positions).astype(np.longdouble)
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    out, at = [], 0
    for axis, n in enumerate(sections):
        phi = p[axis][:, None] * f[None, at:at + n]
        out.append(phi - turn * np.rint(phi / turn))
        at += n
    return np.concatenate(out, axis=1).astype(np.float64)


def pair_channels(R: int, interleaved: bool):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def turn(x, phi, interleaved: bool, sign: float = 1.0) -> np.ndarray:
    a, b = pair_channels(2 * phi.shape[1], interleaved)
    c, s = np.cos(phi)[:, None], sign * np.sin(phi)[:, None]
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def spread(x, phi, interleaved: bool) -> np.ndarray:
    """|x| with both members of a turned pair replaced by the sum of the two: what an
    error of the angle or of a product is measured against."""
    a, b = pair_channels(2 * phi.shape[1], interleaved)
    y = np.abs(np.asarray(x, np.float64))
    both = y[..., a] + y[..., b]
    y[..., a], y[..., b] = both, both
    return y


def rstd(x, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt(np.mean(np.asarray(x, np.float64) ** 2, axis=-1, keepdims=True) + eps)


def forward(x, w, phi, interleaved: bool, eps: float, norm: bool = True):
    """(y, magnitude)."""
    n = np.asarray(x, np.float64)
    if norm:
        n = n * rstd(n, eps) * (1.0 if w is None else w)
    return turn(n, phi, interleaved), spread(n, phi, interleaved)


def backward(dy, x, w, phi, interleaved: bool, eps: float, norm: bool = True):
    """(dx, dw, magnitudes of both)."""
    dy = np.asarray(dy, np.float64)
    g, G = turn(dy, phi, interleaved, -1.0), spread(dy, phi, interleaved)
    if not norm:
        return g, None, G, None
    r = rstd(x, eps)
    n = np.asarray(x, np.float64) * r
    dw, DW = np.sum(g * n, axis=(0, 1)), np.sum(G * np.abs(n), axis=(0, 1))
    w = np.ones(n.shape[-1]) if w is None else w
    t, T = g * w, G * np.abs(w)
    dx = r * (t - n * np.mean(t * n, axis=-1, keepdims=True))
    return dx, dw, r * (T + np.abs(n) * np.mean(T * np.abs(n), axis=-1, keepdims=True)), DW
