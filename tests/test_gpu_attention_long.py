"""GPU: contexts so long that a wave has more than 64 steps of one segment (it then looks up its
pages again) and that the largest number of workgroups is launched, against the fp64
oracle with the bounds of attention_bounds.py.  The table repeats the few pages of a small
cache; some pages, which decide, stand in it once each, anywhere."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from tests import attention_bounds as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
COMMON, ONCE, LENGTHS = 4, 8, [790000, 3, 0, 420019]


class Long:
    def __init__(self, kind, D, Hq, H=8, page=512, seed=0):
        rng = np.random.default_rng([seed, D, Hq, H])
        self.kind, self.D, self.H, self.Hq, self.page = kind, D, H, Hq, page
        pages = COMMON + ONCE
        n, width = pages * page, -(-max(LENGTHS) // page)
        common, at = rng.standard_normal(D), np.arange(n) // page
        q = (rng.standard_normal((len(LENGTHS), Hq, D)) + 2 * common).astype(np.float32)
        k, v = rng.standard_normal((n, H, D)).astype(np.float32), rng.standard_normal((n, H, D)).astype(np.float32)
        # a page that stands once: its scores are some 8 above the others'
        k[at >= COMMON] += (8.0 / (D ** -0.5 * 2 * np.sum(common ** 2)) * common).astype(np.float32)
        v += (0.5 * rng.standard_normal((pages, H, D)))[at].astype(np.float32)
        self.q, self.k, self.v = q, k, v
        self.table = rng.integers(0, COMMON, (len(LENGTHS), width)).astype(np.int32)
        for b, m in enumerate(LENGTHS):
            if m > ONCE * page:
                self.table[b, rng.choice(m // page, ONCE, replace=False)] = COMMON + np.arange(ONCE)
        self.cache = nq.KvCache(pages, H, D, page=page, kind=kind, device=DEV)
        nq.kv_write(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), self.cache, torch.arange(n, device=DEV))

    def run(self, q=BF, y=BF, window=0, table=None):
        self.gq = torch.from_numpy(self.q).to(DEV, q)
        return nq.kv_attention(self.gq, self.cache, torch.from_numpy(self.table if table is None else table).to(DEV),
                               torch.tensor(LENGTHS, dtype=torch.int32, device=DEV), window=window, out_dtype=y)

    def check(self, out, q=BF, y=BF, window=0):
        for b, n in enumerate(LENGTHS):
            got = out[b].double().cpu().numpy()
            if n == 0:
                assert not got.any()
                continue
            t = np.arange(max(0, n - window) if window else 0, n)
            times = np.bincount(self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page,
                                minlength=len(self.k))
            on = times > 0
            want, tol = B.expected(self.gq[b].double().cpu().numpy(), self.k[on], self.v[on], self.kind,
                                   float(np.float32(self.D ** -0.5)), 0, q == F32 or y == F32, y, times[on])
            off = np.abs(got - want)
            assert np.all(off <= tol), (b, float(np.max(off / tol)))


FORMS = [("bf16", 128, 16), ("bf16", 64, 16), ("int8", 128, 16), ("int8", 64, 16), ("int8", 256, 16), ("int4", 64, 16),
         ("int4", 96, 64), ("int4", 128, 64), ("int4", 128, 96), ("int4", 192, 16)]


@pytest.mark.parametrize("kind,D,Hq", FORMS)
@pytest.mark.parametrize("q,y", [(BF, BF), (F32, F32)])
def test_long_contexts(kind, D, Hq, q, y):
    """Shares of some 400 to 600 steps of 32 tokens a workgroup of four waves, one within a
    sequence, some over the border of two; 4 bits of 96 and 128 channels and codes of 64 with
    three workgroups a CU."""
    c = Long(kind, D, Hq)
    c.check(c.run(q, y), q, y)
    c.check(c.run(q, y, window=333333), q, y, 333333)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_more_than_sixteen_query_heads_a_key_head(kind):
    c = Long(kind, 128, 40, H=2, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_a_page_outside_the_cache_far_into_a_sequence(kind):
    """Each alone: where a wave looks up its first pages and where it looks again."""
    c = Long(kind, 64, 16)
    clean = c.run()
    for at in (5, 100, 750, 1540):
        table = c.table.copy()
        table[0, at] = COMMON + ONCE if at % 2 else -1
        out = c.run(table=table)
        assert torch.isnan(out[0]).all() and torch.equal(out[1:], clean[1:])
