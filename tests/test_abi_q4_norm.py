"""C ABI of the 4-bit linears and the block norms: sizes, exports and every
refusal, all on the host (validation happens before any HIP call)."""
import ctypes
import os
import re

import pytest

import binary_rank_gemv_packed_amd as nq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # 256-aligned pointer values that are never dereferenced
GB = 1 << 30
BAD, WS = nq.NQ_ERR_INVALID_ARG, nq.NQ_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nq.LIB_PATH):
        from binary_rank_gemv_packed_amd import build
        build.build()
    return nq.lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nq.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(nq_[a-z0-9_]+)\s*\(", text))
    assert {"nq_q4_pack", "nq_q4_linear_fwd_group", "nq_block_norm_bwd"} <= names
    for name in names:
        assert hasattr(L, name), name


def test_range_status_has_a_text(L):
    assert b"15" in L.nq_status_string(nq.NQ_ERR_RANGE)


# ------------------------------------------------------------------ 4-bit linears
def q4(m=64, n=96, group=32, dt=nq.NQ_F16, zeros=0, blob=FAKE):
    return nq.nq_q4_layer(m, n, group, dt, zeros, blob)


def _bytes(m, n, group, sb, zeros):
    up = lambda v: (v + 255) // 256 * 256
    tiles = ((m + 15) // 16) * ((n + 127) // 128)
    entries = tiles * (128 // group) * 16
    return up(up(up(256 + tiles * 1024) + entries * sb) + (entries if zeros else 0))


@pytest.mark.parametrize("m,n,group,dt,sb,zeros", [(256, 256, 32, nq.NQ_F32, 4, 0), (1, 1, 128, nq.NQ_F16, 2, 1),
                                                   (1100, 4099, 64, nq.NQ_F16, 2, 1),
                                                   (1 << 20, 1 << 20, 32, nq.NQ_F32, 4, 1)])
def test_q4_layer_bytes(L, m, n, group, dt, sb, zeros):
    assert L.nq_q4_layer_bytes(m, n, group, dt, zeros) == _bytes(m, n, group, sb, zeros)


@pytest.mark.parametrize("args", [(0, 8, 32, nq.NQ_F16, 0), (8, (1 << 20) + 1, 32, nq.NQ_F16, 0),
                                  (8, 8, 16, nq.NQ_F16, 0), (8, 8, 256, nq.NQ_F16, 0), (8, 8, 32, nq.NQ_BF16, 0),
                                  (8, 8, 32, nq.NQ_F16, 2), (8, 8, 32, 9, 0)])
def test_q4_layers_out_of_range(L, args):
    assert L.nq_q4_layer_bytes(*args) == 0
    lay = nq.nq_q4_layer(*args, FAKE)
    assert L.nq_q4_pack(ctypes.byref(lay), FAKE + GB, FAKE + GB, None, None) == BAD
    assert L.nq_q4_linear_fwd(ctypes.byref(lay), FAKE, 2, FAKE + GB, 2, 1, None, 0, None) == BAD


def test_q4_pack_refusals(L):
    def pack(lay=None, codes=FAKE + GB, scales=FAKE + 2 * GB, zeros=None):
        return L.nq_q4_pack(ctypes.byref(lay or q4()), codes, scales, zeros, None)
    assert L.nq_q4_pack(None, FAKE, FAKE, None, None) == BAD
    assert pack(q4(blob=0)) == BAD
    assert pack(q4(blob=FAKE + 16)) == BAD
    assert pack(codes=None) == BAD
    assert pack(scales=None) == BAD
    assert pack(scales=FAKE + 2 * GB + 1) == BAD
    assert pack(zeros=FAKE + 3 * GB) == BAD          # zero points for a layer without
    assert pack(q4(zeros=1)) == BAD                  # a layer with zero points, none given
    assert pack(codes=FAKE + 256) == BAD
    assert b"overlap" in L.nq_last_error()
    assert L.nq_q4_unpack(ctypes.byref(q4()), None, None, None) == BAD
    assert L.nq_q4_unpack(ctypes.byref(q4()), FAKE + GB, FAKE + 2 * GB, None) == BAD  # it has no zero points
    assert L.nq_q4_unpack(ctypes.byref(q4()), FAKE, None, None) == BAD


def q4_fwd(L, lay=None, x=FAKE + GB, xdt=nq.NQ_BF16, y=FAKE + 2 * GB, ydt=nq.NQ_BF16, B=1, ws=FAKE + 3 * GB, wsb=GB):
    return L.nq_q4_linear_fwd(ctypes.byref(lay or q4()), x, xdt, y, ydt, B, ws, wsb, None)


def test_q4_forward_refusals(L):
    assert L.nq_q4_linear_fwd(None, FAKE, 2, FAKE + GB, 2, 1, None, 0, None) == BAD
    assert q4_fwd(L, q4(blob=0)) == BAD
    assert q4_fwd(L, B=-1) == BAD
    assert q4_fwd(L, B=(1 << 20) + 1) == BAD
    assert q4_fwd(L, xdt=nq.NQ_F16) == BAD
    assert q4_fwd(L, ydt=nq.NQ_F16) == BAD
    assert q4_fwd(L, x=None) == BAD
    assert q4_fwd(L, y=None) == BAD
    assert q4_fwd(L, x=FAKE + GB + 1) == BAD
    assert q4_fwd(L, y=FAKE + 2 * GB + 2, ydt=nq.NQ_F32) == BAD
    assert q4_fwd(L, y=FAKE + GB + 64) == BAD
    assert b"overlap" in L.nq_last_error()
    assert q4_fwd(L, B=300, wsb=16) == WS
    assert q4_fwd(L, B=300, ws=None) == BAD
    assert q4_fwd(L, B=300, ws=FAKE + 3 * GB + 128) == BAD
    assert q4_fwd(L, B=300, ws=FAKE + 2 * GB) == BAD  # on y
    assert q4_fwd(L, B=300, ws=FAKE + GB) == BAD      # on x
    assert q4_fwd(L, B=0, x=None, y=None) == nq.NQ_OK


def test_q4_workspace(L):
    lay = q4(m=8192, n=28672)
    ref = ctypes.byref(lay)
    assert L.nq_q4_workspace_bytes(None, 1) == 0
    assert L.nq_q4_workspace_bytes(ref, 0) == 0
    assert L.nq_q4_workspace_bytes(ref, 1) == 0
    big = L.nq_q4_workspace_bytes(ref, 2048)
    assert big >= 2 * 2048 * 28672 * 2  # two fp16 images of an fp32 x
    # a bf16 x needs one image only: the stated size covers both types
    assert q4_fwd(L, lay, B=2048, wsb=big // 4) == WS


def test_q4_outputs_on_the_weights(L):
    """An output or a workspace in use that lies on a layer's packed weights."""
    end = L.nq_q4_layer_bytes(q4().m, q4().n, q4().group, q4().scale_dtype, q4().zeros)
    for y in (FAKE, FAKE + end - 2):
        assert q4_fwd(L, y=y) == BAD
        assert b"weights" in L.nq_last_error()
    assert q4_fwd(L, B=300, ws=FAKE) == BAD
    assert b"weights" in L.nq_last_error()
    a, b = q4(m=64), q4(m=32, blob=FAKE + GB)
    for ys in ((FAKE + GB, FAKE + 3 * GB), (FAKE + 3 * GB, FAKE)):  # on the other layer's
        assert L.nq_q4_linear_fwd_group(_group([a, b]), 2, FAKE + 2 * GB, nq.NQ_BF16, (ctypes.c_void_p * 2)(*ys),
                                        nq.NQ_BF16, 1, None, 0, None) == BAD
        assert b"weights" in L.nq_last_error()


def _group(layers):
    return ctypes.cast((ctypes.POINTER(nq.nq_q4_layer) * len(layers))(*[ctypes.pointer(l) for l in layers]),
                       ctypes.c_void_p)


def test_q4_group_refusals(L):
    a, b = q4(m=64), q4(m=32, blob=FAKE + GB)
    ys = (ctypes.c_void_p * 2)(FAKE + 3 * GB, FAKE + 4 * GB)

    def run(layers, count=2, y=ys, x=FAKE + 2 * GB):
        return L.nq_q4_linear_fwd_group(_group(layers), count, x, nq.NQ_BF16, y, nq.NQ_BF16, 1, None, 0, None)
    assert run([a, b], 0) == BAD
    assert run([a, b], nq.NQ_GROUP_MAX + 1) == BAD
    assert L.nq_q4_linear_fwd_group(None, 2, FAKE, 2, ys, 2, 1, None, 0, None) == BAD
    for other in (q4(n=128), q4(group=64), q4(dt=nq.NQ_F32), q4(zeros=1)):
        assert run([a, other]) == BAD
        assert b"shares x" in L.nq_last_error()
        assert L.nq_q4_workspace_bytes_group(_group([a, other]), 2, 300) == 0
    assert run([a, b], y=(ctypes.c_void_p * 2)(FAKE + 3 * GB, FAKE + 3 * GB + 64)) == BAD
    assert run([a, b], y=(ctypes.c_void_p * 2)(FAKE + 3 * GB, None)) == BAD
    assert run([a, b], x=FAKE + 4 * GB) == BAD
    need = L.nq_q4_workspace_bytes_group(_group([a, b]), 2, 300)
    assert need == max(L.nq_q4_workspace_bytes(ctypes.byref(l), 300) for l in (a, b))


# ------------------------------------------------------------------ block norms
def norm(**kw):
    c = dict(d=64, flags=3, act_dtype=nq.NQ_BF16, res_dtype=nq.NQ_F32, param_dtype=nq.NQ_BF16, eps=1e-5, res_scale=1.0,
             block_scale=1.0, weight_offset=0.0, w_post=FAKE, w_pre=FAKE + 4096, gate=None)
    c.update(kw)
    return nq.nq_block_norm(**c)


def fwd(L, n=None, rows=4, h=FAKE + GB, y=FAKE + 2 * GB, gr=None, ho=FAKE + 3 * GB, x=FAKE + 4 * GB, st=FAKE + 5 * GB):
    return L.nq_block_norm_fwd(ctypes.byref(n or norm()), rows, h, y, gr, ho, x, st, None)


NORMS_OUT_OF_RANGE = [dict(d=0), dict(d=nq.NQ_NORM_MAX_DIM + 1), dict(flags=4), dict(act_dtype=nq.NQ_F16),
                      dict(res_dtype=nq.NQ_F16), dict(act_dtype=nq.NQ_F32, res_dtype=nq.NQ_BF16),
                      dict(param_dtype=7), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
                      dict(res_scale=float("inf")), dict(block_scale=float("nan")),
                      dict(weight_offset=float("inf")), dict(w_post=FAKE + 1), dict(gate=FAKE + 3)]


@pytest.mark.parametrize("kw", NORMS_OUT_OF_RANGE)
def test_norms_out_of_range(L, kw):
    assert fwd(L, norm(**kw)) == BAD
    assert L.nq_block_norm_workspace_bytes(ctypes.byref(norm(**kw)), 4) == 0


def test_norm_forward_refusals(L):
    assert L.nq_block_norm_fwd(None, 1, FAKE, FAKE, None, FAKE, FAKE, None, None) == BAD
    assert fwd(L, rows=-1) == BAD
    assert fwd(L, rows=(1 << 20) + 1) == BAD
    assert fwd(L, rows=0, h=None, y=None, ho=None, x=None) == nq.NQ_OK
    assert fwd(L, h=None) == BAD
    assert fwd(L, ho=None) == BAD
    assert fwd(L, x=None) == BAD
    assert fwd(L, norm(flags=1), y=None) == BAD                      # neither a block nor a pre norm
    assert fwd(L, norm(gate=FAKE + 8192), gr=FAKE + 6 * GB) == BAD   # two gates
    assert fwd(L, y=None, gr=FAKE + 6 * GB) == BAD                   # a gate without a block
    assert fwd(L, h=FAKE + GB + 2) == BAD
    assert fwd(L, y=FAKE + 2 * GB + 1) == BAD
    assert fwd(L, st=FAKE + 5 * GB + 2) == BAD
    assert fwd(L, ho=FAKE + GB + 256) == BAD                         # h_out over h, but not h itself
    assert b"overlap" in L.nq_last_error()
    assert fwd(L, x=FAKE + 2 * GB) == BAD                            # x over y
    assert fwd(L, x=FAKE + 3 * GB) == BAD                            # x over h_out
    assert fwd(L, st=FAKE) == BAD                                    # stats over a weight


def bwd(L, n=None, rows=4, dx=FAKE + GB, dho=FAKE + 2 * GB, ho=FAKE + 3 * GB, y=FAKE + 4 * GB, gr=None,
        st=FAKE + 5 * GB, dh=FAKE + 6 * GB, dy=FAKE + 7 * GB, dgr=None, dwp=FAKE + 8 * GB, dwq=FAKE + 9 * GB, dg=None,
        ws=FAKE + 10 * GB, wsb=GB):
    return L.nq_block_norm_bwd(ctypes.byref(n or norm()), rows, dx, dho, ho, y, gr, st, dh, dy, dgr, dwp, dwq, dg, ws,
                               wsb, None)


def test_norm_backward_refusals(L):
    assert bwd(L, rows=-1) == BAD
    assert bwd(L, norm(eps=-1.0)) == BAD
    for kw in (dict(dx=None), dict(ho=None), dict(st=None), dict(dh=None), dict(dy=None)):
        assert bwd(L, **kw) == BAD, kw
    assert bwd(L, gr=FAKE + 11 * GB) == BAD                          # a gate of each row without its gradient
    assert bwd(L, dgr=FAKE + 11 * GB) == BAD
    assert bwd(L, norm(gate=FAKE + 8192), gr=FAKE + 11 * GB, dgr=FAKE + 12 * GB) == BAD
    assert bwd(L, dg=FAKE + 11 * GB) == BAD                          # no channel gate
    assert bwd(L, norm(w_post=None)) == BAD
    assert bwd(L, norm(w_pre=None)) == BAD
    assert bwd(L, norm(flags=2)) == BAD                              # dw_post without a post norm
    assert bwd(L, y=None, dy=None) == BAD                            # dw_post without a block
    assert bwd(L, norm(flags=1), y=None, dwp=None, dwq=None) == BAD  # nothing to do
    assert bwd(L, wsb=16) == WS
    assert bwd(L, ws=None) == BAD
    assert bwd(L, ws=FAKE + 10 * GB + 128) == BAD
    assert bwd(L, dy=FAKE + 4 * GB) == BAD                           # dy over y
    assert bwd(L, dh=FAKE + 2 * GB + 256) == BAD                     # dh over dh_out, but not dh_out itself
    assert bwd(L, dwq=FAKE + 8 * GB) == BAD
    assert bwd(L, ws=FAKE + 3 * GB) == BAD                           # the workspace on h_out
    assert bwd(L, dwp=FAKE + 8 * GB + 2) == BAD
    assert bwd(L, rows=0, dx=None, dho=None, ho=None, y=None, st=None, dh=None, dy=None, dwp=None, dwq=None) == nq.NQ_OK


def test_norm_workspace_grows_with_rows_up_to_the_workgroups(L):
    ref = ctypes.byref(norm(d=100))
    sizes = [L.nq_block_norm_workspace_bytes(ref, r) for r in (1, 2, 100, 1 << 20)]
    assert sizes[0] >= 2 * 100 * 4 and sizes == sorted(sizes) and sizes[-1] <= 2048 * 2 * 100 * 4


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(nq.NQError):
        nq.q4_pack(torch.zeros(4, 8, dtype=torch.uint8), torch.ones(4, 1))
    with pytest.raises(nq.NQError):
        nq.BlockNorm(8, w_pre=torch.ones(8))
    with pytest.raises(nq.NQError):
        nq.block_norm(torch.ones(2, 8), None, nq.BlockNorm(8, act_dtype=torch.float32))
    with pytest.raises(nq.NQError):
        nq.BlockNorm(8, pre=False, w_pre=torch.ones(8))
    with pytest.raises(nq.NQError):
        nq.Q4Group([])
