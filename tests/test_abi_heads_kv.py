"""C ABI and binding of the head norms, the cache of keys and values and the
attention over it: sizes and every refusal, all on the host (validation happens
before any HIP call; pointer values and stand-ins are never dereferenced)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_heads, nq_kv

FAKE = 0x7F0000000000  # 256-aligned
MB = 1 << 20
GB = 1 << 30
BAD, WS = nq.NQ_ERR_INVALID_ARG, nq.NQ_ERR_WORKSPACE
BF, F32, F16 = nq.NQ_BF16, nq.NQ_F32, nq.NQ_F16


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nq.LIB_PATH):
        from binary_rank_gemv_packed_amd import build
        build.build()
    return nq.lib()


def cache(pages=4, heads=2, head_dim=64, page=16, kind=0, data=FAKE):
    return nq.nq_kv_cache(pages, heads, head_dim, page, kind, data)


def norm(head_dim=64, flags=1, act=BF, par=F32, rot=64, axes=1, sections=(32, 0, 0, 0), eps=1e-6, offset=0.0, w_q=FAKE + GB,
         w_k=FAKE + GB + 4096, freq=FAKE + GB + 8192):
    return nq.nq_head_norm(head_dim, flags, act, par, rot, axes, (ctypes.c_int32 * 4)(*sections), eps, offset, w_q, w_k, freq)


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("heads,D,page", [(1, 64, 16), (8, 128, 64), (3, 96, 48), (128, 256, 1024)])
def test_page_bytes(L, heads, D, page):
    up = lambda v: (v + 255) // 256 * 256
    n = heads * page
    assert L.nq_kv_page_bytes(heads, D, page, 0) == up(n * 2 * D * 2)
    assert L.nq_kv_page_bytes(heads, D, page, 1) == up(n * (2 * D + 4))
    assert L.nq_kv_page_bytes(heads, D, page, 2) == up(n * (D + D // 32 * 4))


@pytest.mark.parametrize("args", [(0, 64, 16, 0), (129, 64, 16, 0), (1, 32, 16, 0), (1, 112, 16, 0), (1, 512, 16, 0),
                                  (1, 64, 0, 0), (1, 64, 24, 0), (1, 64, 1040, 0), (1, 64, 16, 3), (1, 64, 16, -1)])
def test_pages_out_of_range(L, args):
    assert L.nq_kv_page_bytes(*args) == 0


def test_workspaces(L):
    assert L.nq_kv_attention_workspace_bytes(ctypes.byref(cache())) % 256 == 0
    assert L.nq_kv_attention_workspace_bytes(ctypes.byref(cache())) > 0
    assert L.nq_kv_attention_workspace_bytes(ctypes.byref(cache(page=17))) == 0
    assert L.nq_kv_attention_workspace_bytes(None) == 0
    assert L.nq_head_norm_workspace_bytes(ctypes.byref(norm()), 100) >= 2 * 64 * 4
    assert L.nq_head_norm_workspace_bytes(ctypes.byref(norm(head_dim=63)), 100) == 0
    assert L.nq_head_norm_workspace_bytes(None, 1) == 0


# ------------------------------------------------------------------ the cache
BAD_CACHES = [dict(pages=0), dict(pages=(1 << 24) + 1), dict(heads=0), dict(heads=129), dict(head_dim=100), dict(page=8),
              dict(page=100), dict(kind=3), dict(data=None), dict(data=FAKE + 128)]


def write(L, c=None, tokens=3, k=FAKE + GB, ks=128, v=FAKE + 2 * GB, vs=128, dtype=BF, slots=FAKE + 3 * GB):
    c = cache() if c is None else c
    return L.nq_kv_write(ctypes.byref(c) if c else None, tokens, k, ks, v, vs, dtype, slots, None)


def read(L, c=None, tokens=3, slots=FAKE + 3 * GB, k=FAKE + GB, v=FAKE + 2 * GB, dtype=BF):
    c = cache() if c is None else c
    return L.nq_kv_read(ctypes.byref(c) if c else None, tokens, slots, k, v, dtype, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_caches_that_are_refused(L, kw):
    c = cache(**kw)
    assert write(L, c) == BAD and read(L, c) == BAD and attend(L, c) == BAD and head_write(L, c=c) == BAD


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(k=None), dict(v=None), dict(slots=None),
                                dict(dtype=F16), dict(dtype=7), dict(k=FAKE + GB + 1), dict(dtype=F32, v=FAKE + 2 * GB + 2),
                                dict(slots=FAKE + 3 * GB + 4), dict(ks=127), dict(vs=0), dict(vs=-128), dict(ks=(1 << 40) + 1),
                                dict(k=FAKE), dict(v=FAKE + 64), dict(slots=FAKE + 8), dict(c=False)])
def test_writes_that_are_refused(L, kw):
    assert write(L, **kw) == BAD
    assert L.nq_last_error()


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(k=None), dict(v=None), dict(slots=None),
                                dict(dtype=F16), dict(k=FAKE + GB + 1), dict(dtype=F32, v=FAKE + 2 * GB + 2),
                                dict(k=FAKE + 2 * GB), dict(v=FAKE + GB + 767), dict(v=FAKE + GB + 766), dict(k=FAKE),
                                dict(v=FAKE + 3 * GB), dict(slots=FAKE + GB + 8), dict(c=False)])
def test_reads_that_are_refused(L, kw):
    assert read(L, **kw) == BAD


def test_nothing_to_do_is_fine(L):
    assert write(L, tokens=0, k=None, v=None, slots=None) == 0
    assert read(L, tokens=0, k=None, v=None, slots=None) == 0
    assert attend(L, B=0, q=None, y=None, table=None, lengths=None, ws=None, ws_bytes=0) == 0
    assert fwd(L, tokens=0, q=None, k=None, q_out=None, k_out=None, pos=None) == 0
    assert head_write(L, tokens=0) == 0
    assert bwd(L, tokens=0, dw_q=None, dw_k=None, ws=None, ws_bytes=0) == 0


# ------------------------------------------------------------------ attention
def attend(L, c=None, B=2, q=FAKE + GB, q_dtype=BF, q_heads=4, table=FAKE + 2 * GB, width=3, lengths=FAKE + 3 * GB, longest=0,
           window=0, scale=0.125, y=FAKE + 4 * GB, y_dtype=BF, ws=FAKE + 5 * GB, ws_bytes=64 * MB):
    c = cache() if c is None else c
    return L.nq_kv_attention(ctypes.byref(c) if c else None, B, q, q_dtype, q_heads, table, width, lengths, longest, window,
                             scale, y, y_dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=1 << 16), dict(q=None), dict(y=None), dict(table=None), dict(lengths=None),
                                dict(ws=None), dict(q_dtype=F16), dict(y_dtype=F16), dict(q_heads=3), dict(q_heads=0),
                                dict(q_heads=1), dict(q_heads=1026), dict(width=0), dict(width=(1 << 26) + 1), dict(longest=-1),
                                dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=FAKE + GB + 1),
                                dict(y=FAKE + 4 * GB + 8), dict(table=FAKE + 2 * GB + 2), dict(lengths=FAKE + 3 * GB + 1),
                                dict(ws=FAKE + 5 * GB + 128), dict(y=FAKE + GB), dict(y=FAKE), dict(ws=FAKE), dict(ws=FAKE + GB),
                                dict(y=FAKE + 2 * GB + 16), dict(y=FAKE + 3 * GB), dict(ws=FAKE + 4 * GB), dict(c=False),
                                dict(B=(1 << 16) - 1, width=1 << 26, table=FAKE + 64 * GB, q=FAKE + 1024 * GB * 32,
                                     y=FAKE + 1024 * GB * 34, lengths=FAKE + 1024 * GB * 36, ws=FAKE + 1024 * GB * 38)])
def test_attentions_that_are_refused(L, kw):
    assert attend(L, **kw) == BAD
    assert L.nq_last_error()


def test_attention_workspace_too_small(L):
    need = L.nq_kv_attention_workspace_bytes(ctypes.byref(cache()))
    assert attend(L, ws_bytes=need - 1) == WS


# ------------------------------------------------------------------ head norms
def fwd(L, N=None, tokens=5, q=FAKE, qs=256, qh=4, k=FAKE + MB, ks=128, kh=2, pos=FAKE + 2 * MB, q_out=FAKE + 3 * MB,
        k_out=FAKE + 4 * MB):
    N = norm() if N is None else N
    return L.nq_head_norm_fwd(ctypes.byref(N) if N else None, tokens, q, qs, qh, k, ks, kh, pos, q_out, k_out, None)


def head_write(L, N=None, c=None, tokens=5, q=FAKE + 16 * MB, qs=256, qh=4, k=FAKE + 17 * MB, ks=128, v=FAKE + 18 * MB, vs=128,
               pos=FAKE + 19 * MB, slots=FAKE + 20 * MB, q_out=FAKE + 21 * MB):
    N, c = norm() if N is None else N, cache() if c is None else c
    return L.nq_head_norm_kv_write(ctypes.byref(N), tokens, q, qs, qh, k, ks, v, vs, pos, ctypes.byref(c) if c else None,
                                   slots, q_out, None)


def bwd(L, N=None, tokens=5, dq_out=FAKE, dk_out=FAKE + MB, q=FAKE + 2 * MB, qs=256, qh=4, k=FAKE + 3 * MB, ks=128, kh=2,
        pos=FAKE + 4 * MB, dq=FAKE + 5 * MB, dk=FAKE + 6 * MB, dw_q=FAKE + 7 * MB, dw_k=FAKE + 8 * MB, ws=FAKE + 9 * MB,
        ws_bytes=8 * MB):
    N = norm() if N is None else N
    return L.nq_head_norm_bwd(ctypes.byref(N) if N else None, tokens, dq_out, dk_out, q, qs, qh, k, ks, kh, pos, dq, dk, dw_q,
                              dw_k, ws, ws_bytes, None)


BAD_NORMS = [dict(head_dim=0), dict(head_dim=63), dict(head_dim=514), dict(flags=4), dict(act=F16), dict(act=9), dict(par=3),
             dict(rot=-2), dict(rot=63), dict(rot=66), dict(flags=0, rot=0, sections=(0, 0, 0, 0)), dict(axes=0), dict(axes=5),
             dict(sections=(31, 0, 0, 0)), dict(axes=2, sections=(33, -1, 0, 0)), dict(axes=2, sections=(32, 1, 0, 0)),
             dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(offset=float("nan")), dict(w_q=FAKE + 2),
             dict(par=F16, w_k=FAKE + 1), dict(freq=None), dict(freq=FAKE + 4)]


@pytest.mark.parametrize("kw", BAD_NORMS)
def test_norms_that_are_refused(L, kw):
    N = norm(**kw)
    assert fwd(L, N) == BAD and bwd(L, N) == BAD and head_write(L, N) == BAD


@pytest.mark.parametrize("kw", [dict(N=False), dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(qh=-1), dict(kh=1025),
                                dict(qh=0, kh=0), dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(pos=None),
                                dict(pos=FAKE + 2 * MB + 4), dict(q=FAKE + 1), dict(k_out=FAKE + 4 * MB + 1), dict(qs=255),
                                dict(ks=0), dict(q_out=FAKE, qs=257), dict(q_out=FAKE + 512), dict(k_out=FAKE),
                                dict(q_out=FAKE + 4 * MB), dict(q_out=FAKE + 2 * MB), dict(k_out=FAKE + GB),
                                dict(k_out=FAKE + GB + 8192)])
def test_forwards_that_are_refused(L, kw):
    assert fwd(L, **kw) == BAD
    assert L.nq_last_error()


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(qh=-1), dict(q=None), dict(k=None), dict(v=None), dict(slots=None),
                                dict(pos=None), dict(q_out=None), dict(vs=127), dict(v=FAKE + 18 * MB + 1),
                                dict(slots=FAKE + 20 * MB + 4), dict(c=False), dict(N=norm(head_dim=96, rot=0, sections=(0,) * 4)),
                                dict(q_out=FAKE), dict(v=FAKE), dict(slots=FAKE), dict(q_out=FAKE + 18 * MB),
                                dict(q=FAKE, q_out=FAKE), dict(c=cache(data=FAKE + 16 * MB))])
def test_head_writes_that_are_refused(L, kw):
    assert head_write(L, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(N=False), dict(tokens=-1), dict(qh=0, kh=0), dict(dq_out=None), dict(dk_out=None),
                                dict(q=None), dict(k=None), dict(dq=None), dict(dk=None), dict(pos=None), dict(ws=None),
                                dict(ws=FAKE + 9 * MB + 128), dict(dw_q=FAKE + 7 * MB + 2), dict(N=norm(w_q=None)),
                                dict(N=norm(w_k=None)), dict(N=norm(flags=0)), dict(dq=FAKE + MB), dict(dq=FAKE + 2 * MB),
                                dict(dk=FAKE + 5 * MB), dict(dw_k=FAKE + 7 * MB), dict(ws=FAKE), dict(dw_q=FAKE + GB),
                                dict(qs=200), dict(ks=-1)])
def test_backwards_that_are_refused(L, kw):
    assert bwd(L, **kw) == BAD


def test_backward_workspace_too_small(L):
    assert bwd(L, ws_bytes=255) == WS


# ------------------------------------------------------------------ the binding
GPU = torch.device("cuda", 0)


class Stand:
    """What the binding asks of a tensor that lies on a GPU."""

    def __init__(self, shape, dtype, device=GPU, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        whole = torch.empty(shape, device="meta").stride()
        self._stride = whole if stride is None else stride
        self._contiguous = self._stride == whole
        self.is_cuda = device.type == "cuda"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return FAKE

    def double(self):
        return Stand(self.shape, torch.float64, self.device)

    def contiguous(self):
        return self


T_BF, T_F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8
CPU, OTHER = torch.device("cpu"), torch.device("cuda", 1)


def held_cache(kind="bf16"):
    return nq.KvCache(4, 2, 64, page=16, kind=kind, into=Stand((4, nq.lib().nq_kv_page_bytes(2, 64, 16, nq.KV_KINDS[kind])), U8))


def refuses(call, *args, **kw):
    with pytest.raises(nq.NQError):
        call(*args, **kw)


def test_binding_caches():
    held_cache()
    for kw in (dict(kind="fp8"), dict(page=20), dict(head_dim=65), dict(heads=0), dict(pages=0)):
        refuses(nq.KvCache, **{**dict(pages=4, heads=2, head_dim=64, page=16, kind="bf16"), **kw})
    for into in (Stand((4, 100), U8), Stand((4, 8192), torch.int8), Stand((4, 8192), U8, CPU), Stand((4, 8192), U8, stride=(9000, 1))):
        refuses(nq.KvCache, 4, 2, 64, page=16, into=into)


def test_binding_cache_calls():
    c, k, s = held_cache(), Stand((3, 2, 64), T_BF), Stand((3,), I64)
    for bad in (Stand((3, 2, 64), torch.float16), Stand((3, 3, 64), T_BF), Stand((3, 2, 32), T_BF), Stand((3, 128), T_BF),
                Stand((3, 2, 64), T_BF, CPU), Stand((3, 2, 64), T_BF, OTHER), Stand((3, 2, 64), T_BF, stride=(128, 1, 2)),
                Stand((3, 2, 64), T_BF, stride=(256, 128, 1))):
        refuses(nq.kv_write, bad, k, c, s)
        refuses(nq.kv_write, k, bad, c, s)
    refuses(nq.kv_write, k, Stand((3, 2, 64), T_F32), c, s)
    refuses(nq.kv_write, k, Stand((4, 2, 64), T_BF), c, s)
    for bad in (Stand((4,), I64), Stand((3,), I32), Stand((3,), I64, CPU), Stand((3,), I64, stride=(2,)), Stand((3, 1), I64)):
        refuses(nq.kv_write, k, k, c, bad)
    for bad in (Stand((3,), I32), Stand((3,), I64, CPU), Stand((3, 1), I64)):
        refuses(nq.kv_read, c, bad)
    refuses(nq.kv_read, c, s, torch.float16)


def test_binding_attention():
    c, q, t, n, ws = held_cache(), Stand((2, 4, 64), T_BF), Stand((2, 3), I32), Stand((2,), I32), Stand((64 * MB,), U8)
    y = Stand((2, 4, 64), T_BF)
    ok = dict(q=q, cache=c, table=t, lengths=n, y=y, workspace=ws)
    for kw in (dict(q=Stand((2, 4, 64), torch.float16)), dict(q=Stand((2, 256), T_BF)), dict(q=Stand((2, 4, 96), T_BF)),
               dict(q=Stand((2, 4, 64), T_BF, CPU)), dict(q=Stand((2, 4, 64), T_BF, stride=(512, 64, 1))),
               dict(y=Stand((2, 4, 64), torch.float16)), dict(y=Stand((3, 4, 64), T_BF)), dict(table=Stand((2,), I32)),
               dict(table=Stand((3, 3), I32)), dict(table=Stand((2, 3), I64)), dict(table=Stand((2, 3), I32, stride=(6, 1))),
               dict(lengths=Stand((2,), I64)), dict(lengths=Stand((3,), I32)), dict(lengths=Stand((2,), I32, OTHER)),
               dict(workspace=Stand((MB,), T_F32)), dict(workspace=Stand((MB,), U8, CPU))):
        refuses(nq.kv_attention_into, **{**ok, **kw})


def test_binding_head_norms():
    w, f = Stand((64,), T_F32), Stand((32,), torch.float64)
    for kw in (dict(w_q=Stand((63,), T_F32)), dict(w_k=Stand((64,), T_BF)), dict(w_q=Stand((64,), T_F32, CPU), w_k=None),
               dict(act_dtype=torch.float16), dict(norm=False), dict(inv_freq=Stand((32,), T_F32, OTHER)),
               dict(inv_freq=Stand((2, 16), T_F32)), dict(sections=(16, 15)), dict(sections=(8,) * 5), dict(sections=()),
               dict(sections=(40, -8))):
        refuses(nq.HeadNorm, **{**dict(head_dim=64, w_q=w, w_k=w, inv_freq=f), **kw})
    N = nq.HeadNorm(64, w_q=w, w_k=w, inv_freq=f, sections=(16, 16))
    q, k, p = Stand((5, 4, 64), T_BF), Stand((5, 2, 64), T_BF), Stand((2, 5), I64)
    assert N.check(q, k, p)[1:6] == (5, 4, 256, 2, 128)
    assert N.check(Stand((5, 4, 64), T_BF, stride=(600, 64, 1)), None, p)[3] == 600
    for args in ((None, None, p), (Stand((5, 4, 64), T_F32), k, p), (q, Stand((4, 2, 64), T_BF), p), (q, Stand((5, 2, 32), T_BF), p),
                 (Stand((5, 256), T_BF), k, p), (Stand((5, 4, 64), T_BF, CPU), None, p), (q, k, None), (q, k, Stand((5,), I64)),
                 (q, k, Stand((2, 5), I32)), (q, k, Stand((2, 5), I64, CPU)), (q, k, Stand((2, 5), I64, stride=(10, 1))),
                 (Stand((5, 4, 64), T_BF, stride=(600, 1, 4)), k, p)):
        refuses(nq.head_norm, *args, N)
    refuses(nq.head_norm, Stand((5, 4, 64), T_BF, stride=(600, 64, 1)), k, p, N, inplace=True)
    c, v, s = held_cache(), Stand((5, 2, 64), T_BF), Stand((5,), I64)
    for kw in (dict(v=Stand((5, 3, 64), T_BF)), dict(v=Stand((4, 2, 64), T_BF)), dict(v=Stand((5, 2, 64), T_F32)),
               dict(slots=Stand((4,), I64)), dict(k=Stand((5, 4, 64), T_BF), v=Stand((5, 4, 64), T_BF)), dict(k=None)):
        refuses(nq.head_norm_write, **{**dict(q=q, k=k, v=v, positions=p, norm=N, cache=c, slots=s), **kw})
    for kw in (dict(dq=None), dict(dk=None), dict(dq=Stand((5, 4, 64), T_F32)), dict(dk=Stand((5, 4, 64), T_BF)), dict(k=None),
               dict(dq=Stand((5, 4, 64), T_BF, stride=(600, 64, 1))), dict(workspace=Stand((MB,), T_F32))):
        refuses(nq.head_norm_backward, **{**dict(dq=q, dk=k, q=q, k=k, positions=p, norm=N), **kw})


# ------------------------------------------------------------------ the oracles
def test_oracle_codes():
    """Codes and scales by hand: ties to even, the scale rounded to bf16."""
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :5] = [127, 0.5, 1.5, -2.5, 126.5]
    assert nq_kv.scales(x, "int8")[0, 0, 0] == 1
    assert list(nq_kv.codes(x, "int8")[0, 0, :5]) == [127, 0, 2, -2, 126]
    x[0, 0, 32:35] = [7, -3.5, 0.25]
    assert list(nq_kv.scales(x, "int4")[0, 0]) == [float(nq_kv.bf16(np.float32(127) / np.float32(7))), 1]
    assert list(nq_kv.held(x, "int4")[0, 0, 32:35]) == [7, -4, 0]
    x[0, 0, 40] = np.inf
    assert np.isnan(nq_kv.held(x, "int4")[0, 0, 32:]).all() and not np.isnan(nq_kv.held(x, "int4")[0, 0, :32]).any()
    assert np.isnan(nq_kv.held(x, "int8")).all()
    assert nq_kv.bf16(np.float32(1.00390625)) == 1 and nq_kv.bf16(np.float32(1.01171875)) == np.float32(1.015625)


def test_oracle_attention_is_a_weighted_mean():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    y, _, _ = nq_kv.attention(q, k, v, 0.0)
    assert np.allclose(y[0], v[:, 0].mean(0)) and np.allclose(y[3], v[:, 1].mean(0))
    y, _, _ = nq_kv.attention(q, k, v, 0.7, window=1)
    assert np.allclose(y[1], v[4, 0]) and np.allclose(y[2], v[4, 1])
    assert not nq_kv.attention(q, k[:0], v[:0], 1.0)[0].any()
    a = nq_kv.attention(q, k, v, 0.5)[0]
    w = np.exp(0.5 * (k[:, 0] @ q[0]))
    assert np.allclose(a[0], (w[:, None] * v[:, 0]).sum(0) / w.sum())


def test_oracle_rotation_keeps_lengths_and_adds_up():
    rng = np.random.default_rng(2)
    x, f = rng.standard_normal((3, 2, 10)), 10.0 ** -np.arange(3)
    for interleaved in (False, True):
        phi = nq_heads.angles(np.array([[1, 7, 100000], [5, 0, 2]]), f, (1, 2))
        y = nq_heads.turn(x, phi, interleaved)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1)) and np.array_equal(y[..., 6:], x[..., 6:])
        assert np.allclose(nq_heads.turn(y, phi, interleaved, -1.0), x)
    assert np.allclose(np.cos(phi[:, 0]), np.cos([1, 7, 100000])) and np.allclose(np.sin(phi[:, 1]), np.sin([0.5, 0, 0.2]))
    a, b = nq_heads.pair_channels(6, False)
    assert list(b - a) == [3, 3, 3] and list(nq_heads.pair_channels(6, True)[1]) == [1, 3, 5]


def test_oracle_gradients_are_slopes():
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((4, 2, 12)), rng.standard_normal((4, 2, 12)), rng.standard_normal(12)
    phi = nq_heads.angles(rng.integers(0, 50, (1, 4)), 3.0 ** -np.arange(4), (4,))
    dx, dw, _, _ = nq_heads.backward(dy, x, w, phi, False, 1e-5)
    loss = lambda x, w: float(np.sum(dy * nq_heads.forward(x, w, phi, False, 1e-5)[0]))
    way, step = rng.standard_normal(x.shape), 1e-6
    assert abs((loss(x + step * way, w) - loss(x - step * way, w)) / (2 * step) - np.sum(dx * way)) < 1e-6
    way = rng.standard_normal(12)
    assert abs((loss(x, w + step * way) - loss(x, w - step * way)) / (2 * step) - np.sum(dw * way)) < 1e-6


def test_layout_has_a_place_for_every_value():
    """The documented layout (nq_kv.h) written out here: each byte of a tile's keys and
    values belongs to one slot alone, and all are used."""
    def byte(lane, b, lane_bytes):
        whole, rest = lane_bytes & ~15, lane_bytes & 15
        return (b >> 4) * 1024 + lane * 16 + (b & 15) if b < whole else (whole >> 4) * 1024 + lane * rest + b - whole

    for D in (64, 96, 128, 192, 256):
        for bits in (16, 8, 4):
            lane_bytes, half = D * bits // 32, 2 * D * bits
            keys, values = {}, {}
            for slot in range(16):
                for c in range(D):
                    i, g, e = c // 32, c % 32 // 8, c % 8
                    for n in range(max(1, bits // 8)):
                        b = 16 * i + 2 * e + n if bits == 16 else 8 * i + e if bits == 8 else 4 * i + [0, 2, 0, 2, 1, 3, 1, 3][e]
                        keys.setdefault(byte(slot + 16 * g, b, lane_bytes), set()).add(slot)
                        x, lane = c // 16, c % 16 + 16 * (slot // 4)
                        j = slot % 4
                        b = 8 * x + 2 * j + n if bits == 16 else 4 * x + j if bits == 8 else 4 * i + [0, 2, 1, 3][j]
                        values.setdefault(byte(lane, b, lane_bytes), set()).add(slot)
            for places in (keys, values):
                assert set(places) == set(range(half)) and all(len(s) == 1 for s in places.values())
