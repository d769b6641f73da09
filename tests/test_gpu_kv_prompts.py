"""GPU: prompts of the cache, whose tokens are written and read four at a time, at every head
size: bit for bit the oracle's values, and byte for byte what the same tokens leave when
they come a few at a call."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_kv as O
from tests.test_gpu_kv import DIMS, KINDS, check, read, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def scattered(rng, n, T):
    """T slots of n: runs that begin and end anywhere, in any order, single slots, some left out."""
    free = rng.permutation(n // 64)
    out = []
    for block in free:
        lo, hi = rng.integers(0, 20), rng.integers(40, 65)
        run = np.arange(block * 64 + lo, block * 64 + hi)
        out.append(rng.permutation(run) if block % 5 == 0 else run)
        out.append(rng.choice([-1, -7, n, n + 64], rng.integers(0, 3)))
        if sum(map(len, out)) >= T:
            break
    slots = np.concatenate(out)[:T].astype(np.int64)
    assert len(slots) == T
    return torch.from_numpy(slots)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,page,n,T", [(64, 48, 10 * 48, 257), (5, 16, 340 * 16, 3301)])
def test_prompts(kind, D, dtype, H, page, n, T):
    """More than 16384 heads of tokens: a number of heads that is no power of two, a last group
    of four that is not full, slots in runs, single and left out, over an older filling."""
    rng = np.random.default_rng([21, D, H])
    cache = nq.KvCache(n // page, H, D, page=page, kind=kind, device=DEV)
    twin = nq.KvCache(n // page, H, D, page=page, kind=kind, device=DEV)
    cache.data.fill_(0xFF), twin.data.fill_(0xFF)
    everywhere = torch.arange(n, device=DEV)
    k, v = (tokens(rng, n, H, D, dtype) for _ in range(2))
    nq.kv_write(k.to(DEV), v.to(DEV), cache, everywhere)
    check(cache, everywhere, k, v)
    few = 16383 // H
    for lo in range(0, n, few):
        nq.kv_write(k[lo:lo + few].to(DEV), v[lo:lo + few].to(DEV), twin, everywhere[lo:lo + few])
    assert torch.equal(cache.data, twin.data)
    slots = scattered(rng, n, T)
    assert T * H >= 16384 and T % 4
    nk, nv = (tokens(rng, T, H, D, dtype) for _ in range(2))
    nq.kv_write(nk.to(DEV), nv.to(DEV), cache, slots.to(DEV))
    on = (slots >= 0) & (slots < n)
    k[slots[on]], v[slots[on]] = nk[on], nv[on]
    check(cache, everywhere, k, v)
    for out in (F32, BF):
        for got, x in zip(read(cache, slots.to(DEV), out), (k, v)):
            want = O.held(x[slots[on]].float().numpy(), kind)
            if out == BF:
                want = O.bf16(want.astype(np.float32)).astype(np.float64)
            assert np.array_equal(got[on.numpy()], want) and not got[~on.numpy()].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", DIMS)
def test_prompts_whose_values_are_not_finite(kind, D):
    """Infinities and NaN in some tokens of a group of four stay in their token's group of
    channels."""
    rng = np.random.default_rng([22, D])
    H, n = 64, 320
    cache = nq.KvCache(n // 16, H, D, page=16, kind=kind, device=DEV)
    k, v = (tokens(rng, n, H, D, F32) for _ in range(2))
    for x in (k, v):
        for value in (float("inf"), float("-inf"), float("nan"), 0.0):
            x[rng.integers(0, n, 40), rng.integers(0, H, 40), rng.integers(0, D, 40)] = value
        x[rng.integers(0, n, 5)] = 0.0
    slots = torch.arange(n, device=DEV)
    nq.kv_write(k.to(DEV), v.to(DEV), cache, slots)
    check(cache, slots, k, v)
