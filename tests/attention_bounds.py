"""How far one token's attention over the cache may be from the fp64 oracle: bounds for
each kind of cache and form, derived and not fitted, and emulations of what they have to
reject.

With e = 2^-24, x the scores, P the softmax's weights, M = sum P |v| over held values:
  scores    D products, exact, summed in fp32, times scale: off by (D + 16) e X at most, X the largest
            scale * sum |q k| of a head (fp32 queries come as three pieces, of which the second
            and third add 2^-7 to a sum's size).  4 bits with bf16 q and y: codes enter as c + 24 or
            c + 136, so that each 32 channels' product and what is taken off again are rounded,
            up to 32 times each, at the size of scale s sum 144 |q|: 64 e of that.
  weights   off by d = the scores' error, and 2^-22 for the subtraction and the exponential; the
            sum of n weights by n / 32 + 64 roundings.  Numerator and denominator: twice d + 2^-22.
  rounding  bf16 q and y: a weight (codes: weight times scale) comes as two bf16 pieces of 8
            significant bits, half a step 2^-8 each, so it is off by 2^-16; over 4 bits as one, off by
            2^-8.  fp32 q or y: three pieces, off by 2^-23 at most.
  values    4 bits with bf16 q and y: as the scores, 64 e of sum P s 144.
  output    half a step of its type."""
from __future__ import annotations

import numpy as np
import torch

from oracle import nq_kv as O

E = 2.0 ** -24


def softmax(q, k, scale, times=None):
    """(heads, n) weights and largest scale * sum |q k| of a head, q (Hq, D), k (n, H, D), token t
    there times[t] times."""
    H = k.shape[1]
    r = q.shape[0] // H
    x = np.concatenate([scale * (q[h * r:(h + 1) * r] @ k[:, h].T) for h in range(H)])
    big = np.concatenate([abs(scale) * (np.abs(q[h * r:(h + 1) * r]) @ np.abs(k[:, h]).T) for h in range(H)])
    p = np.exp(x - x.max(axis=1, keepdims=True)) * (1.0 if times is None else times)
    return p / p.sum(axis=1, keepdims=True), big.max(axis=1, keepdims=True)


def mix(p, v):
    """sum over tokens of p (Hq, n) times v (n, H, D)."""
    r = p.shape[0] // v.shape[1]
    return np.concatenate([p[h * r:(h + 1) * r] @ v[:, h] for h in range(v.shape[1])])


def expected(q, k, v, kind, scale, window=0, fine=False, out=torch.float32, times=None):
    """(values, bound) of one sequence: q (Hq, D) as the call has it, k and v (n, H, D) fp32 as
    they were written; times: how often it has each token (once)."""
    q = np.asarray(q, np.float64)
    if window:
        k, v = k[max(0, len(k) - window):], v[max(0, len(v) - window):]
    H, D = k.shape[1:]
    n = len(k) if times is None else int(np.sum(times))
    hk, hv = O.held(k, kind), O.held(v, kind)
    p, big = softmax(q, hk, scale, times)
    y, mag = mix(p, hv), mix(p, np.abs(hv))
    d = (D + 16) * E * big
    bias = 0.0
    if kind == "int4" and not fine:
        r, size = q.shape[0] // H, lambda s: np.repeat(s.astype(np.float64), 32, axis=-1)
        sk, sv = size(O.scales(k, kind)), size(O.scales(v, kind))
        d = d + 64 * E * 144 * abs(scale) * np.concatenate(
            [(np.abs(q[h * r:(h + 1) * r]) @ sk[:, h].T).max(axis=1, keepdims=True) for h in range(H)])
        bias = 64 * E * 144 * mix(p, sv)
    w = 2.0 ** -23 if fine else 2.0 ** -8 if kind == "int4" else 2.0 ** -16
    tol = (2 * (2 * d + 2.0 ** -22) + w + (n / 32 + 64) * E) * mag + bias
    return y, tol + torch.finfo(out).eps / 2 * (np.abs(y) + tol) + 1e-42


def emulate(q, k, v, kind, scale, round_q=False, round_p=False):
    """The formula with queries or weights rounded to one bf16 piece."""
    q = O.bf16(q).astype(np.float64) if round_q else np.asarray(q, np.float64)
    hk, hv = O.held(k, kind), O.held(v, kind)
    p, _ = softmax(q, hk, scale)
    if round_p:
        p = O.bf16(p.astype(np.float32)).astype(np.float64)
        p /= p.sum(axis=1, keepdims=True)
    return mix(p, hv)


def sequence(rng, n, H, D, loud=1.0, Hq=8, few=6):
    """Queries, keys and values: normal, values not about zero.  The queries of a key head have a
    direction in common, and `few` tokens anywhere a score about 12 above the others: what is
    lost of a score or weight is then not evened out over many tokens."""
    common = np.repeat(rng.standard_normal((H, D)), Hq // H, axis=0)
    q = loud * (rng.standard_normal((Hq, D)) + 2 * common)
    k = rng.standard_normal((n, H, D))
    up = rng.choice(n, min(few, n), replace=False)
    k[up] += 12.0 / (D ** -0.5 * loud * 2 * D) * common[::Hq // H]
    v = rng.standard_normal((n, H, D)) + 0.25
    return q.astype(np.float32), k.astype(np.float32), v.astype(np.float32)
