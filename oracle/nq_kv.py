"""fp64 oracle of the paged cache of keys and values and of one token's attention
over it.

held(x, kind): what the cache stands for where x was written; attention(): softmax
of the scores of the tokens that are seen, with the magnitudes that rounding is
measured against.
"""
from __future__ import annotations

import numpy as np

MOST = {"int8": 127, "int4": 7}


def bf16(x) -> np.ndarray:
    """x to the nearest bf16 value, ties to even (x fp32 or exactly representable in it)."""
    x = np.asarray(x, np.float32)
    u = x.view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32))


def groups(D: int, kind: str) -> int:
    return {"bf16": 0, "int8": 1, "int4": D // 32}[kind]


def scales(x, kind: str) -> np.ndarray:
    """(..., groups): bf16(max |x| / most), the quotient in fp32; NaN for a group with
    an infinity or a NaN."""
    x = np.asarray(x, np.float32)
    n = groups(x.shape[-1], kind)
    g = x.reshape(*x.shape[:-1], n, x.shape[-1] // n)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.max(np.abs(g), axis=-1)
        return np.where(np.isfinite(top), bf16(top / np.float32(MOST[kind])), np.float32(np.nan))


def codes(x, kind: str) -> np.ndarray:
    x, s = np.asarray(x, np.float32), scales(x, kind)
    g = x.reshape(*s.shape, x.shape[-1] // s.shape[-1])
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(s[..., None] > 0, g / s[..., None], np.float32(0))
    return np.clip(np.rint(np.nan_to_num(c)), -MOST[kind], MOST[kind]).reshape(x.shape)


def held(x, kind: str) -> np.ndarray:
    """(..., heads, D) fp32 -> fp64 values of the cache."""
    if kind == "bf16":
        return bf16(x).astype(np.float64)
    s, c = scales(x, kind).astype(np.float64), codes(x, kind)
    return (c.reshape(*s.shape, c.shape[-1] // s.shape[-1]) * s[..., None]).reshape(c.shape)


def attention(q, k, v, scale: float, window: int = 0):
    """q (Hq, D), k and v (n, H, D) of one sequence -> (y, sum of p |v|, largest
    scale * sum |q k| of a head's tokens), (Hq, D), (Hq, D) and (Hq, 1)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, H, D = k.shape
    if window:
        k, v = k[max(0, n - window):], v[max(0, n - window):]
    r = q.shape[0] // H
    y, mag, big = np.zeros(q.shape), np.zeros(q.shape), np.zeros((q.shape[0], 1))
    if len(k) == 0:
        return y, mag, big
    for h in range(H):
        at = slice(h * r, (h + 1) * r)
        x = scale * (q[at] @ k[:, h].T)
        p = np.exp(x - x.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        y[at], mag[at] = p @ v[:, h], p @ np.abs(v[:, h])
        big[at] = abs(scale) * (np.abs(q[at]) @ np.abs(k[:, h]).T).max(axis=1, keepdims=True)
    return y, mag, big
