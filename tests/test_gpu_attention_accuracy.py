"""GPU: what each form of the attention promises of its arithmetic, on inputs where a few tokens
decide: fp32 q or y as good as three bf16 pieces for every kind of cache, 4 bits without
an allowance for codes that fp32 forms do not shift.  test_attention_bounds.py shows that the
bounds reject less."""
import numpy as np
import pytest
import torch

from tests import attention_bounds as B
from tests.test_attention_bounds import DIMS, KINDS, LOUD, case
from tests.test_gpu_attention_range import attend

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(seqs, kind, q, y, **kw):
    D = seqs[0][1].shape[2]
    scale = float(np.float32(D ** -0.5))
    if q == BF:
        seqs = [(B.O.bf16(s[0]), s[1], s[2]) for s in seqs]
    got = attend(seqs, kind, q, y, scale=scale, **kw)
    for y_b, (qs, k, v) in zip(got, seqs):
        want, tol = B.expected(qs, k, v, kind, scale, fine=q == F32 or y == F32, out=y)
        off = np.abs(y_b - want)
        assert np.all(off <= tol), (len(k), float(np.max(off / tol)))


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("loud", LOUD)
@pytest.mark.parametrize("q,y", [(F32, F32), (BF, F32), (F32, BF), (BF, BF)])
def test_forms(D, kind, loud, q, y):
    """One launch, and the same sequences beside a longer one; up to eight query heads a key
    head and more."""
    check([case(D, loud, n) for n in (33, 400)], kind, q, y, max_length=400)
    check([case(D, loud, n) for n in (33, 400, 2300)], kind, q, y)
    check([case(D, loud, n, Hq=24) for n in (400, 2300)], kind, q, y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q,y", [(F32, F32), (BF, BF)])
def test_more_than_sixteen_query_heads_a_key_head(kind, q, y):
    check([case(128, 1.0, n, 1, 40) for n in (33, 400, 2300)], kind, q, y)
