"""fp64 oracle of the norms between two blocks and of their gradients.

    u  = y ry wp, ry = (mean y^2 + eps)^-1/2    h' = a h + b gate u    x = h' rh wq, rh = (mean h'^2 + eps)^-1/2

wp, wq: the norms' weights plus their offset (None: that norm is left out);
gate: broadcast against (rows, d), or None.
"""
from __future__ import annotations

import numpy as np


def rstd(v, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt(np.mean(np.asarray(v, np.float64) ** 2, axis=1, keepdims=True) + eps)


def forward(h, y, wp, wq, gate, a: float, b: float, eps: float, post: bool = True, pre: bool = True):
    """(h', x or None)."""
    h = np.asarray(h, np.float64)
    if y is not None:
        u = np.asarray(y, np.float64)
        if post:
            u = u * rstd(u, eps) * (1.0 if wp is None else wp)
        h = a * h + b * (1.0 if gate is None else gate) * u
    return h, (h * rstd(h, eps) * (1.0 if wq is None else wq) if pre else None)


def backward(dx, dh, h_out, y, wp, wq, gate, a: float, b: float, ry, rh, post: bool = True, pre: bool = True):
    """Gradients from those of x and h', with the norms' 1/rms (rows x 1) given.
    A dict; "gate" is the gradient of a gate of each row and channel, "w_post",
    "w_pre" the sums over rows, "M" the magnitudes that rounding is measured
    against (the same formulas with every term's absolute value)."""
    g = np.zeros(h_out.shape) if dh is None else np.asarray(dh, np.float64)
    G = np.abs(g)
    out, M = {}, {}
    ones = np.ones(h_out.shape[1])
    wp, wq = (ones if w is None else w for w in (wp, wq))
    if pre:
        hn, dx = h_out * rh, np.asarray(dx, np.float64)
        t = dx * wq
        g = g + rh * (t - hn * np.mean(t * hn, axis=1, keepdims=True))
        G = G + rh * (np.abs(t) + np.abs(hn) * np.mean(np.abs(t * hn), axis=1, keepdims=True))
        out["w_pre"], M["w_pre"] = np.sum(dx * hn, axis=0), np.sum(np.abs(dx * hn), axis=0)
    if y is None:
        return {**out, "h": g, "M": {**M, "h": G}}
    out["h"], M["h"] = a * g, abs(a) * G
    v, V = b * g, abs(b) * G
    yn = y * ry if post else np.asarray(y, np.float64)
    gate = 1.0 if gate is None else gate
    out["gate"], M["gate"] = v * yn * (wp if post else 1.0), V * np.abs(yn * (wp if post else 1.0))
    s, S = v * gate, V * np.abs(gate)
    out["w_post"], M["w_post"] = np.sum(s * yn, axis=0), np.sum(S * np.abs(yn), axis=0)
    if post:
        s, S = s * wp, S * np.abs(wp)
        S = ry * (S + np.abs(yn) * np.mean(S * np.abs(yn), axis=1, keepdims=True))
        s = ry * (s - yn * np.mean(s * yn, axis=1, keepdims=True))
    out["y"], M["y"] = s, S
    return {**out, "M": M}
