"""The bounds that the attention is held to reject what they are there to reject: on the same
inputs as the GPU tests, queries or weights in one bf16 piece where three are due, no output,
the plain mean, keys or values with one wrong code, an excess of the 4-bit codes that is left in."""
import numpy as np
import pytest

from oracle import nq_kv as O
from tests import attention_bounds as B

DIMS, KINDS = [64, 96, 128, 192, 256], ["bf16", "int8", "int4"]
LOUD = [0.25, 1.0, 4.0]  # size of the queries
N = [33, 400, 2300]


def case(D, loud, n, H=2, Hq=8):
    return B.sequence(np.random.default_rng([D, int(8 * loud), n, Hq]), n, H, D, loud, Hq)


def rejected(bad, want, tol):
    return bool(np.any(np.abs(bad - want) > tol))


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("loud", LOUD)
@pytest.mark.parametrize("n", N)
def test_what_is_rejected(D, kind, loud, n):
    q, k, v = case(D, loud, n)
    scale = float(np.float32(D ** -0.5))
    want, tol = B.expected(q, k, v, kind, scale, fine=True)
    hk, hv = O.held(k, kind), O.held(v, kind)
    _, size = B.expected(q, k, v, kind, scale, fine=False, out=B.torch.bfloat16)
    mag = B.mix(B.softmax(q.astype(np.float64), hk, scale)[0], np.abs(hv))
    most = mag.max(axis=1, keepdims=True)
    assert np.all(tol <= 0.01 * most) and np.all(size <= (0.05 if loud <= 1 else 0.2) * most)
    assert rejected(B.emulate(q, k, v, kind, scale, round_q=True), want, tol)
    if loud <= 1:  # above it a weight's half step is less than the scores' roundings
        assert rejected(B.emulate(q, k, v, kind, scale, round_p=True), want, tol)
    bq = O.bf16(q)
    low, wide = B.expected(bq, k, v, kind, scale, fine=False, out=B.torch.bfloat16)
    p, _ = B.softmax(bq.astype(np.float64), hk, scale)
    mean = np.repeat(hv.mean(axis=0), q.shape[0] // hv.shape[1], axis=0)
    for w, t in ((want, tol), (low, wide)):
        assert rejected(np.zeros_like(w), w, t)
        assert rejected(mean, w, t)
    if kind != "int4" and loud < 1:
        assert rejected(O.bf16(B.emulate(bq, k, v, kind, scale, round_p=True).astype(np.float32)), low, wide)
    if kind == "int4":  # codes 8 too large, keys' or values'
        more = lambda x: O.held(x, kind) + 8 * np.repeat(O.scales(x, kind).astype(np.float64), 32, axis=-1)
        assert rejected(B.mix(B.softmax(bq.astype(np.float64), more(k), scale)[0], hv), low, wide)
        assert rejected(B.mix(p, more(v)), low, wide)
    if kind != "bf16" and n == 33:  # the likeliest token's value one code off in one channel
        t = int(np.argmax(p[0]))
        off = hv.copy()
        off[t, 0, 5] += float(O.scales(v, kind)[t, 0, 0])
        assert rejected(B.mix(B.softmax(q.astype(np.float64), hk, scale)[0], off), want, tol)
