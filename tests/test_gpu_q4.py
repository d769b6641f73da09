"""GPU: linears with 4-bit weights against the fp64 oracle.

Tolerance (derived, not fitted).  With M = sum_j |W[i, j] x[b, j]|, every product
is exact for bf16 x; the sums hold at most n + 32 roundings of partial sums that
M bounds, taken at 2^-23 each (an MFMA may truncate); fp32 x adds 2^-22 M for its
two fp16 pieces, and parts under 2^-39 of the largest of a row are dropped.  A
worst case of n roundings that all add up does not happen for more than a few
terms: the bound taken is the longest chain of one element, 128 sums in a group
(256 for two pieces), one a group and one for each of up to 16 waves or 32 splits.
A bf16 output adds half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_q4 as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def make(m, n, B, G, zeros, scale, x_dtype, seed=0):
    rng = np.random.default_rng([seed, m, n, B, G, zeros])
    ng = -(-n // G)
    q = rng.integers(0, 16, (m, n)).astype(np.uint8)
    s = torch.from_numpy(rng.standard_normal((m, ng)).astype(np.float32)).to(DT[scale])
    z = rng.integers(0, 16, (m, ng)).astype(np.uint8) if zeros else None
    x = torch.from_numpy(rng.standard_normal((B, n)).astype(np.float32)).to(DT[x_dtype])
    return q, s, z, x


def pack(q, s, z, G):
    return nq.q4_pack(torch.from_numpy(q).to(DEV), s.to(DEV), torch.from_numpy(z).to(DEV) if z is not None else None,
                      group=G)


def f64(t):
    return t.double().cpu().numpy()


def check(y, x, q, s, z, G):
    """Every output of y within the bound; returns the largest share of it."""
    n = q.shape[1]
    ref, M = Q.linear(f64(x), q, f64(s), z, G), Q.magnitude(f64(x), q, f64(s), z, G)
    P = 2 if x.dtype == torch.float32 else 1
    chain = 128 * P + -(-n // G) + 32
    tol = chain * 2.0 ** -23 * M + (2.0 ** -22 * M if P == 2 else 0.0)
    tol = tol + 2.0 ** -39 * np.abs(f64(x)).max(1, keepdims=True) * np.abs(Q.weight(q, f64(s), z, G)).sum(1)
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(f64(y) - ref)
    share = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    assert share <= 1.0, share
    return share


SHAPES = [(1, 1), (16, 128), (17, 129), (63, 17), (256, 256), (100, 300), (300, 520), (33, 2179), (1100, 4099), (40, 8200)]


# ------------------------------------------------------------------ packing
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("G,zeros,scale", [(32, True, "f16"), (64, False, "f32"), (128, True, "f32")])
def test_pack_round_trip(m, n, G, zeros, scale):
    q, s, z, _ = make(m, n, 1, G, zeros, scale, "bf16")
    layer = pack(q, s, z, G)
    codes, zz = nq.q4_unpack(layer)
    assert np.array_equal(codes.cpu().numpy(), q)
    assert (zz is None) if z is None else np.array_equal(zz.cpu().numpy(), z)


def test_blob_as_documented():
    """Header, tile layout and group entries, read byte by byte as the layout says."""
    m, n, G = 37, 300, 64
    q, s, z, _ = make(m, n, 1, G, True, "f16", "bf16")
    blob = pack(q, s, z, G).blob.cpu().numpy()
    head = blob[:72].view(np.uint32)
    assert list(head[:7]) == [0x3134514E, 1, m, n, G, nq.NQ_F16, 1] and head[7] == 0
    off_codes, off_scales, off_zeros, total = blob[32:64].view(np.uint64)
    assert total == blob.size
    KT, SG = 3, 2
    words = blob[int(off_codes):int(off_scales)].view(np.uint32)
    for rt in range(3):
        for kt in range(KT):
            for lane in range(64):
                for t in range(4):
                    w = int(words[((rt * KT + kt) * 64 + lane) * 4 + t])
                    for p in range(8):
                        i = 16 * rt + (lane & 15)
                        j = 128 * kt + 32 * t + 8 * (lane >> 4) + (2 * p if p < 4 else 2 * (p - 4) + 1)
                        assert (w >> (4 * p)) & 15 == (q[i, j] if i < m and j < n else 0)
    sc = blob[int(off_scales):int(off_scales) + 3 * KT * SG * 32].view(np.float16).reshape(3, KT, 4, SG, 4)
    zz = blob[int(off_zeros):int(off_zeros) + 3 * KT * SG * 16].reshape(3, KT, 16, SG)
    for i in range(48):
        for g in range(KT * SG):
            inside = i < m and g < s.shape[1]
            rt, r, kt, gg = i // 16, i % 16, g // SG, g % SG
            assert sc[rt, kt, r // 4, gg, r % 4] == (s[i, g].numpy() if inside else 0)
            assert zz[rt, kt, r, gg] == (z[i, g] if inside else 0)


@pytest.mark.parametrize("where", ["code", "zero"])
def test_pack_refuses_values_above_15(where):
    q, s, z, _ = make(20, 70, 1, 32, True, "f16", "bf16")
    (q if where == "code" else z)[19, 2] = 16
    with pytest.raises(nq.NQError) as e:
        pack(q, s, z, 32)
    assert e.value.status == nq.NQ_ERR_RANGE


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("B", [1, 3, 16])
@pytest.mark.parametrize("G,zeros,scale,xd", [(32, True, "f32", "f32"), (32, False, "f16", "bf16"),
                                              (64, True, "f16", "bf16"), (64, False, "f32", "f32"),
                                              (128, True, "f16", "f32"), (128, False, "f32", "bf16")])
def test_decode_parity(m, n, B, G, zeros, scale, xd):
    q, s, z, x = make(m, n, B, G, zeros, scale, xd)
    layer = pack(q, s, z, G)
    for yd in (torch.float32, torch.bfloat16):
        check(nq.q4_linear(x.to(DEV), layer, out_dtype=yd), x, q, s, z, G)


@pytest.mark.parametrize("m,n", [(1, 1), (17, 129), (130, 300), (300, 2179), (520, 1024)])
@pytest.mark.parametrize("B", [17, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("G,zeros,scale,xd", [(32, True, "f32", "f32"), (64, True, "f16", "bf16"),
                                              (128, False, "f16", "f32"), (128, False, "f16", "bf16")])
def test_batches_and_prompts(m, n, B, G, zeros, scale, xd):
    q, s, z, x = make(m, n, B, G, zeros, scale, xd)
    layer = pack(q, s, z, G)
    for yd in (torch.float32, torch.bfloat16):
        check(nq.q4_linear(x.to(DEV), layer, out_dtype=yd), x, q, s, z, G)


@pytest.mark.parametrize("B", [1, 2, 4, 5, 7, 8, 9, 12, 15])
def test_every_small_batch(B):
    for xd in ("bf16", "f32"):
        q, s, z, x = make(200, 700, B, 64, True, "f16", xd)
        check(nq.q4_linear(x.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32), x, q, s, z, 64)


@pytest.mark.parametrize("m,n,B", [(8192, 1024, 2), (9000, 500, 16), (8200, 4096, 70), (4096, 11008, 1)])
def test_long_and_wide(m, n, B):
    q, s, z, x = make(m, n, B, 128, True, "f16", "bf16")
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, 128), out_dtype=torch.float32), x, q, s, z, 128)


@pytest.mark.parametrize("m,n,B,xd", [(64, 28672, 16, "bf16"), (2100, 28672, 2, "f32"), (5000, 16384, 9, "f32"),
                                      (300, 28672, 3, "bf16"), (130, 28672, 70, "bf16"), (4100, 8192, 5, "bf16"),
                                      (2000, 9000, 1, "bf16")])
def test_columns_split_and_shared(m, n, B, xd):
    """Row lengths and batches on both sides of what a workgroup holds of x."""
    for G, zeros in ((128, True), (32, False)):
        q, s, z, x = make(m, n, B, G, zeros, "f16", xd)
        layer = pack(q, s, z, G)
        need = nq.q4_workspace_bytes(layer, B)
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
        y = torch.full((B, m), float("nan"), device=DEV)
        check(nq.q4_linear_into(x.to(DEV), layer, y, ws), x, q, s, z, G)
        assert bool((ws[need:] == 0xFF).all())


def test_a_layer_twice_in_a_group():
    q, s, z, x = make(100, 300, 4, 64, True, "f16", "bf16")
    layer = pack(q, s, z, 64)
    a, b, c = nq.q4_linear_group(x.to(DEV), [layer, layer, layer], out_dtype=torch.float32)
    assert torch.equal(a, b) and torch.equal(a, c)
    check(a, x, q, s, z, 64)


@pytest.mark.parametrize("B", [1, 4, 16, 40, 200])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_whole_numbers_are_exact(B, G, xd):
    """Whole x below 2^7 and scales that are powers of two: every partial sum is a
    whole number below 2^24 steps, so that nothing rounds."""
    m, n = 150, 390
    q, s, z, _ = make(m, n, B, G, True, "f16", xd, seed=5)
    rng = np.random.default_rng([5, B])
    s = torch.from_numpy(2.0 ** rng.integers(-1, 2, s.shape)).half()
    x = torch.from_numpy(rng.integers(-60, 61, (B, n)).astype(np.float32)).to(DT[xd])
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, G), out_dtype=torch.float32)
    assert np.array_equal(f64(y), Q.linear(f64(x), q, f64(s), z, G))


@pytest.mark.parametrize("B", [1, 5, 200])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-120, -40, 40, 100])
def test_far_magnitudes(B, xd, power):
    q, s, z, x = make(64, 300, B, 64, True, "f32", xd)
    x = (x.double() * 2.0 ** power).to(DT[xd])
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32), x, q, s, z, 64)


@pytest.mark.parametrize("B", [1, 6, 130])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_magnitudes_that_differ_within_a_row(B, xd):
    q, s, z, x = make(64, 520, B, 32, True, "f32", xd)
    x = (x.double() * 2.0 ** torch.from_numpy(np.random.default_rng(6).integers(-30, 31, 520))).to(DT[xd])
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, 32), out_dtype=torch.float32), x, q, s, z, 32)


@pytest.mark.parametrize("B", [3, 20, 130])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_row(B, xd, value):
    q, s, z, x = make(70, 300, B, 64, True, "f16", xd)
    bad = x.clone()
    bad[1, 299] = value
    layer = pack(q, s, z, 64)
    y, ref = nq.q4_linear(bad.to(DEV), layer, out_dtype=torch.float32), nq.q4_linear(x.to(DEV), layer, out_dtype=torch.float32)
    assert not torch.isfinite(y[1]).any()
    keep = [b for b in range(B) if b != 1]
    assert torch.equal(y[keep], ref[keep])
    if value != value:
        return
    # an infinity times a weight that is not zero, all else finite: an infinity of that sign
    w = Q.weight(q, f64(s), z, 64)[:, 299]
    some = torch.from_numpy(w != 0)
    assert torch.equal(y[1].cpu()[some], torch.from_numpy(np.sign(w) * value)[some].float())


def test_small_scales():
    """fp16 scales below its normal numbers keep their value."""
    q, s, z, x = make(40, 300, 3, 64, True, "f16", "bf16")
    s = (s.float() * 2.0 ** -20).half()
    assert bool((s.abs() < 2.0 ** -14).all()) and bool((s != 0).any())
    for B in (3, 70):
        xx = x[:1].expand(B, -1).contiguous()
        check(nq.q4_linear(xx.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32), xx, q, s, z, 64)


def test_zero_rows_and_zero_scales():
    q, s, z, x = make(40, 200, 3, 32, True, "f16", "bf16")
    s[:, 2] = 0
    x[1] = 0
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, 32), out_dtype=torch.float32)
    check(y, x, q, s, z, 32)
    assert not y[1].any()


# ------------------------------------------------------------------ groups
@pytest.mark.parametrize("ms", [(300, 64, 64), (700, 700), (17, 1, 100, 1500), (8192, 1024, 1024)])
@pytest.mark.parametrize("B", [1, 4, 16, 30, 100])
def test_groups_equal_their_layers(ms, B):
    n, G = 520, 64
    sets = [make(m, n, B, G, True, "f16", "bf16", seed=i) for i, m in enumerate(ms)]
    x = sets[0][3]
    layers = [pack(q, s, z, G) for q, s, z, _ in sets]
    ys = nq.q4_linear_group(x.to(DEV), layers, out_dtype=torch.float32)
    for (q, s, z, _), y in zip(sets, ys):
        check(y, x, q, s, z, G)


# ------------------------------------------------------------------ memory
@pytest.mark.parametrize("B", [1, 5, 70])
@pytest.mark.parametrize("off", [1, 3, 8])
@pytest.mark.parametrize("yd", [torch.float32, torch.bfloat16])
def test_unaligned_tensors_and_what_lies_round_them(B, off, yd):
    m, n, G = 131, 136, 64
    for xd in ("bf16", "f32"):
        q, s, z, x = make(m, n, B, G, True, "f16", xd)
        xb = torch.full((B * n + 2 * off,), float("nan"), dtype=x.dtype, device=DEV)
        xb[off:off + B * n] = x.to(DEV).view(-1)
        yb = torch.full((B * m + 2 * off,), 7.0, dtype=yd, device=DEV)
        layer = pack(q, s, z, G)
        need = nq.q4_workspace_bytes(layer, B)
        ws = torch.full((max(need, 256) + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        y = nq.q4_linear_into(xb[off:off + B * n].view(B, n), layer, yb[off:off + B * m].view(B, m), ws)
        check(y, x, q, s, z, G)
        assert bool((yb[:off] == 7).all()) and bool((yb[off + B * m:] == 7).all())
        assert bool((ws[max(need, 256):] == 0xA5).all())


def test_repeated_calls_give_identical_bits():
    for B in (1, 16, 200):
        q, s, z, x = make(520, 4099, B, 32, True, "f16", "bf16")
        layer, xd = pack(q, s, z, 32), x.to(DEV)
        first = nq.q4_linear(xd, layer, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(nq.q4_linear(xd, layer, out_dtype=torch.float32), first)


def test_single_rows_and_empty_batches():
    q, s, z, x = make(40, 200, 2, 32, False, "f16", "bf16")
    layer = pack(q, s, z, 32)
    two = nq.q4_linear(x.to(DEV), layer)
    one = nq.q4_linear(x[0].to(DEV), layer)
    assert one.shape == (40,) and two.dtype == torch.bfloat16
    check(one[None], x[:1], q, s, z, 32)
    assert nq.q4_linear(x[:0].to(DEV), layer).shape == (0, 40)
    wide = torch.randn(2, 400, device=DEV).to(torch.bfloat16)[:, ::2]  # not contiguous: copied
    assert torch.equal(nq.q4_linear(wide, layer), nq.q4_linear(wide.contiguous(), layer))


def test_on_another_stream():
    q, s, z, x = make(300, 2179, 200, 64, True, "f16", "bf16")
    layer, xd = pack(q, s, z, 64), x.to(DEV)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    y = nq.q4_linear(xd, layer, out_dtype=torch.float32, stream=stream)
    # a temporary of the call must not be handed out again while the stream uses it
    junk = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(8)]
    stream.synchronize()
    check(y, x, q, s, z, 64)
    del junk


def test_binding_refusals():
    q, s, z, x = make(40, 200, 2, 32, True, "f16", "bf16")
    layer, x = pack(q, s, z, 32), x.to(DEV)
    codes, scales, zeros = torch.from_numpy(q).to(DEV), s.to(DEV), torch.from_numpy(z).to(DEV)
    y, ws = torch.empty(2, 40, device=DEV), nq.new_q4_workspace(layer, 2)
    for bad in (lambda: nq.q4_pack(codes.int(), scales, zeros, 32),
                lambda: nq.q4_pack(codes, scales.double(), zeros, 32),
                lambda: nq.q4_pack(codes, scales[:, :-1], zeros, 32),
                lambda: nq.q4_pack(codes, scales, zeros[:-1], 32),
                lambda: nq.q4_pack(codes, scales, zeros, 48),
                lambda: nq.q4_linear(x.half(), layer),
                lambda: nq.q4_linear(x[:, :-1], layer),
                lambda: nq.q4_linear(x.cpu(), layer),
                lambda: nq.q4_linear(x, layer, out_dtype=torch.float16),
                lambda: nq.q4_linear_into(x, layer, y.t(), ws),
                lambda: nq.q4_linear_into(x, layer, y[:, :-1], ws),
                lambda: nq.q4_linear_into(x[:, ::2], layer, y, ws),
                lambda: nq.q4_linear_into(x, layer, y, ws.cpu()),
                lambda: nq.q4_linear_group_into(x, [layer], [y, y], ws),
                lambda: nq.q4_linear_group_into(x, [layer, layer], [y, y], ws)):
        with pytest.raises(nq.NQError):
            bad()
