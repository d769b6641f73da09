"""GPU: attention of large batches that are cut into shares: more units than shares, where a
unit is joined by the first border in it, against the fp64 oracle with the bounds of
attention_bounds.py.  Sequences share the pages of one small cache."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from tests import attention_bounds as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
PAGE, PAGES, WIDTH = 32, 120, 100


class Shared:
    """A cache of PAGES pages, and sequences over any of them in any order."""

    def __init__(self, H, D, kind, seed=0):
        rng = np.random.default_rng([seed, H, D])
        n = PAGES * PAGE
        self.H, self.D, self.kind = H, D, kind
        self.k, self.v = (rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2))
        self.v += 0.25
        self.cache = nq.KvCache(PAGES, H, D, page=PAGE, kind=kind, device=DEV)
        nq.kv_write(torch.from_numpy(self.k).to(DEV), torch.from_numpy(self.v).to(DEV), self.cache, torch.arange(n, device=DEV))

    def check(self, lengths, Hq, q=BF, y=BF, window=0, some=40, seed=1):
        rng = np.random.default_rng([seed, len(lengths), Hq])
        n = len(lengths)
        table = rng.integers(0, PAGES, (n, WIDTH)).astype(np.int32)
        gq = torch.randn((n, Hq, self.D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(q)
        ws = nq.new_kv_workspace(n, Hq, self.cache)
        ws.fill_(0xFF)
        out = torch.full((n, Hq, self.D), 77.0, device=DEV, dtype=y)
        gt, gl = torch.from_numpy(table).to(DEV), torch.from_numpy(lengths.astype(np.int32)).to(DEV)
        nq.kv_attention_into(gq, self.cache, gt, gl, out, ws, window=window)
        bad, none = (lengths < 0) | (lengths > WIDTH * PAGE), lengths == 0
        got = out.double().cpu().numpy()
        assert np.isnan(got[bad]).all() and not got[none].any() and np.isfinite(got[~bad]).all()
        assert torch.equal(nq.kv_attention(gq, self.cache, gt, gl, window=window, out_dtype=y, workspace=ws).view(torch.uint8),
                           out.view(torch.uint8))
        live = np.flatnonzero(~bad & ~none)
        rows = set(rng.choice(live, min(some, len(live)), replace=False)) | set(live[np.argsort(lengths[live])[-6:]]) | {live[0], live[-1]}
        for b in sorted(rows):
            t = np.arange(lengths[b])
            at = table[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE
            want, tol = B.expected(gq[b].double().cpu().numpy(), self.k[at], self.v[at], self.kind,
                                   float(np.float32(self.D ** -0.5)), window, q == F32 or y == F32, y)
            off = np.abs(got[b] - want)
            assert np.all(off <= tol), (b, lengths[b], float(np.max(off / tol)))


def mixed(n, seed=0, long=12):
    """Mostly short, some without tokens, a few bad, `long` of some thousand anywhere."""
    rng = np.random.default_rng([n, seed])
    lengths = rng.integers(0, 70, n)
    lengths[rng.random(n) < 0.2] = 0
    lengths[rng.random(n) < 0.03] = -4
    lengths[rng.random(n) < 0.03] = WIDTH * PAGE + 1
    lengths[rng.choice(n, long, replace=False)] = rng.integers(1500, WIDTH * PAGE + 1, long)
    lengths[0], lengths[-1] = 65, WIDTH * PAGE
    return lengths


@pytest.mark.parametrize("n", [65, 96, 257, 1000, 4097])
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("D,Hq", [(64, 8), (96, 40), (128, 64)])
def test_mixed_lengths(n, kind, D, Hq):
    """8 key heads: 520 units and more."""
    Shared(8, D, kind).check(mixed(n), Hq)


@pytest.mark.parametrize("kind,D,q,y", [("bf16", 192, BF, BF), ("int8", 256, BF, F32), ("int4", 128, F32, F32),
                                        ("int4", 256, BF, BF), ("bf16", 256, F32, BF)])
def test_other_forms(kind, D, q, y):
    Shared(2, D, kind).check(mixed(600), 6, q, y)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_more_than_sixteen_query_heads_a_key_head(kind):
    Shared(1, 128, kind).check(mixed(900), 40)


@pytest.mark.parametrize("window", [1, 33, 1700])
def test_windows(window):
    Shared(4, 64, "bf16").check(mixed(500), 8, window=window)


def test_all_long_all_short_and_hardly_any():
    """Every border in a unit of its own, several borders in one, and none at all."""
    s = Shared(8, 64, "int8")
    s.check(np.full(300, 700), 8)
    s.check(np.full(90, 3100), 8)
    s.check(np.ones(700, np.int64), 8)
    few = np.zeros(900, np.int64)
    few[450] = 3000
    s.check(few, 8)
    few[[3, 898]] = 3200, 33
    s.check(few, 8)


def test_the_most_sequences_a_call_may_have():
    Shared(2, 64, "int4").check(mixed(65535, long=30), 4, F32, F32)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_captured_and_replayed_while_sequences_come_and_go(kind):
    """One captured call of a large batch over lengths that change between the replays, on a
    workspace that eager calls use in between."""
    s = Shared(8, 64, kind)
    n = 200
    rng = np.random.default_rng(3)
    q = torch.randn((n, 8, 64), device=DEV).bfloat16()
    table = torch.from_numpy(rng.integers(0, PAGES, (n, WIDTH)).astype(np.int32)).to(DEV)
    lengths, ws, out = torch.zeros(n, dtype=torch.int32, device=DEV), nq.new_kv_workspace(n, 8, s.cache), torch.empty_like(q)
    side = torch.cuda.Stream()

    def call():
        return nq.kv_attention_into(q, s.cache, table, lengths, out, ws)
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for now in (mixed(n, 1), mixed(n, 2), np.zeros(n), np.full(n, WIDTH * PAGE), np.ones(n), mixed(n, 3)):
        lengths.copy_(torch.from_numpy(now.astype(np.int32)))
        want = call().clone()
        ws.fill_(0xFF), out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))
