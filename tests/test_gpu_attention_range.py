"""GPU: attention over large values: finite wherever n |v| is (for 4 bits with bf16 q and y
(n + 700) |v|), whatever the order in which the scores come, against the fp64 oracle with
the bounds of attention_bounds.py."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from tests import attention_bounds as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rising(n, D, seed, up, large):
    """One sequence whose scores, in powers of two, go from 0 to `up` in its last half, with
    values near `large`.  Channel 0 carries the scores."""
    rng = np.random.default_rng([n, D, seed])
    q = np.zeros((8, D), np.float32)
    q[:, 0] = 1.0
    k = rng.standard_normal((n, 2, D)).astype(np.float32)
    k[..., 0] = 0.0
    k[n // 2:, :, 0] = up
    v = (large * rng.uniform(0.5, 1.0, (n, 2, D))).astype(np.float32)
    return q, k, v


def attend(seqs, kind, q, y, page=32, scale=float(np.log(2.0)), **kw):
    H, D = seqs[0][1].shape[1:]
    need = [-(-len(s[1]) // page) for s in seqs]
    cache = nq.KvCache(sum(need), H, D, page=page, kind=kind, device=DEV)
    cache.data.fill_(0xFF)
    table = np.zeros((len(seqs), max(need)), np.int32)
    slots, at = [], 0
    for b, (_, k, _) in enumerate(seqs):
        table[b, :need[b]] = np.arange(at, at + need[b])
        slots.append(np.arange(len(k)) + at * page)
        at += need[b]
    k, v = (torch.from_numpy(np.concatenate([s[i] for s in seqs])).to(DEV) for i in (1, 2))
    nq.kv_write(k, v, cache, torch.from_numpy(np.concatenate(slots)).to(DEV))
    lengths = torch.tensor([len(s[1]) for s in seqs], dtype=torch.int32, device=DEV)
    out = nq.kv_attention(torch.from_numpy(np.stack([s[0] for s in seqs])).to(DEV, q), cache, torch.from_numpy(table).to(DEV),
                          lengths, scale=scale, out_dtype=y, **kw)
    return out.double().cpu().numpy()


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,y", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [600, 2600])
def test_large_values(kind, D, q, y, n):
    """Scores that rise by 7.5 after a wave's first pairs, in one launch and in two; values near
    3.4e38 / (n + 700)."""
    fine = q == F32
    large = 3.0e38 / (n + 700)
    seqs = [rising(n, D, 0, 7.5, large), rising(n - 37, D, 1, 7.5, -large), rising(n, D, 2, -7.5, large)]
    got = attend(seqs, kind, q, y)
    for y_b, (qs, k, v) in zip(got, seqs):
        want, tol = B.expected(qs, k, v, kind, float(np.float32(np.log(2.0))), fine=fine, out=y)
        assert np.all(np.isfinite(y_b))
        assert np.all(np.abs(y_b - want) <= tol), float(np.max(np.abs(y_b - want) / tol))


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("q,y", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("large", [1e-28, 1e-20, 1.0, 1e30])
def test_any_size_of_values(kind, q, y, large):
    seqs = [rising(700, 64, 3, up, large) for up in (7.5, 30.0, -30.0, 100.0)]
    got = attend(seqs, kind, q, y)
    for y_b, (qs, k, v) in zip(got, seqs):
        want, tol = B.expected(qs, k, v, kind, float(np.float32(np.log(2.0))), fine=q == F32, out=y)
        assert np.all(np.abs(y_b - want) <= tol), float(np.max(np.abs(y_b - want) / tol))


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("n", [600, 2600])
def test_scores_of_any_size(kind, n):
    """Scores around 2^28, where fp32 steps are 16 and more: parts of a sequence that hold
    different maxima are weighed against each other as the formula does."""
    qs, k, v = rising(n, 64, 4, 0.0, 1.0)
    k[:, :, 1:] = 0.0
    k[:, :, 0] = 1.0
    k[n // 3:2 * n // 3, :, 0] = 0.5
    seqs = [((up * qs).astype(np.float32), k, v) for up in (2.0 ** 28, -2.0 ** 28, 2.0 ** 27, 2.0 ** 31)]
    got = attend(seqs, kind, F32, F32)
    for y_b, (q0, k0, v0) in zip(got, seqs):
        p, _ = B.softmax(q0.astype(np.float64), B.O.held(k0, kind), 1.0)
        hv = B.O.held(v0, kind)
        want, mag = B.mix(p, hv), B.mix(p, np.abs(hv))  # weights are 1 and 0: the sums' roundings alone
        assert np.all(np.abs(y_b - want) <= (n / 32 + 80) * B.E * mag)
