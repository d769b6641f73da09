"""GPU: 4-bit linears on every path (columns shared or split, prompts in tiles of 64
or 128 columns, with and without K splits) where an error would average out under
a worst-case bound: the second fp16 image of fp32 activations, and the partial sums
of groups of several layers."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_q4 as Q
from tests.test_gpu_q4 import DEV, DT, check, f64, make, pack

pytestmark = pytest.mark.gpu

# shared: one row, several; split: few row tiles, many; prompts: up to 64 rows, more,
# with K splits (a small m and a large n) and without
PATHS = [(200, 8200, 1), (300, 1100, 3), (1100, 4099, 7), (2100, 28672, 2), (64, 28672, 16), (500, 16384, 9),
         (130, 9000, 20), (130, 9000, 64), (130, 9000, 65), (700, 300, 20), (4100, 700, 200)]


@pytest.mark.parametrize("m,n,B", PATHS)
@pytest.mark.parametrize("G,zeros", [(32, True), (64, False), (128, True)])
def test_the_remainders_of_fp32_activations_are_exact(m, n, B, G, zeros):
    """Whole x of up to 17 bits: an fp16 piece holds 11 of them and the remainder's
    piece the others.  Sixteen columns of a row of W are 1 or -1 times a scale of 1/2, 1
    or 2, the others 0, so that every partial sum is a multiple of 1/2 of at most
    16 x 2^17 x 2 = 2^22: nothing rounds, and y is the exact result.  Without the
    remainders at least nine of ten outputs would differ (checked on the oracle)."""
    rng = np.random.default_rng([11, m, n, B, G])
    ng = -(-n // G)
    z = rng.integers(1, 15, (m, ng)) if zeros else np.full((m, ng), 8)
    q = np.repeat(z, G, axis=1)[:, :n]
    k = min(16, n)
    at = np.argsort(rng.random((m, n)), axis=1)[:, :k] if n < 2000 else rng.integers(0, n, (m, k))
    np.put_along_axis(q, at, np.take_along_axis(q, at, 1) + rng.choice([-1, 1], (m, k)), 1)
    q = q.astype(np.uint8)
    s = torch.from_numpy(2.0 ** rng.integers(-1, 2, (m, ng))).half()
    x = torch.from_numpy((rng.integers(2 ** 16, 2 ** 17, (B, n)) * rng.choice([-1, 1], (B, n))).astype(np.float32))
    zz = z.astype(np.uint8) if zeros else None
    want = Q.linear(f64(x), q, f64(s), zz, G)
    assert np.abs(want).max() < 2.0 ** 23
    one_piece = Q.linear(f64((x / 2 ** 3).half()) * 2 ** 3, q, f64(s), zz, G)
    assert np.mean(one_piece != want) > 0.9
    y = nq.q4_linear(x.to(DEV), pack(q, s, zz, G), out_dtype=torch.float32)
    assert np.array_equal(f64(y), want)


@pytest.mark.parametrize("m,n,B", PATHS)
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_relative_error(m, n, B, xd):
    """Rounding errors of independent signs add as a root of their count: with the
    chain of at most 128 P + groups + 32 sums at 2^-23 of sums of the size of
    sqrt(sum (W x)^2), and 2^-22 of each product for the two pieces of an fp32 x, the
    relative L2 error of y (whose own size is that root) is at most
    2^-23 sqrt(chain) + 2^-22.  A lost remainder costs about 2^-13."""
    G = 64
    q, s, z, x = make(m, n, B, G, True, "f16", xd)
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, G), out_dtype=torch.float32)
    w = Q.weight(q, f64(s), z, G)
    size = np.sqrt(np.sum((f64(x) ** 2) @ (w ** 2).T))
    chain = 128 * (2 if xd == "f32" else 1) + -(-n // G) + 32
    assert np.linalg.norm(f64(y) - f64(x) @ w.T) <= (2.0 ** -23 * chain ** 0.5 + 2.0 ** -22) * size


@pytest.mark.parametrize("ms,n,B", [((300, 17, 100), 9000, 5), ((300, 17, 100), 9000, 16), ((17, 2100, 1, 40), 16384, 9),
                                    ((5000, 130), 28672, 16), ((130, 700), 4099, 20), ((130, 700), 4099, 130),
                                    ((700, 130, 33), 9000, 65)])
@pytest.mark.parametrize("xd,G,zeros", [("bf16", 128, True), ("f32", 32, False), ("f32", 64, True)])
def test_groups_with_split_columns(ms, n, B, xd, G, zeros):
    """Layers of unlike heights: partial sums of each at its place in the workspace,
    which starts as NaN and is not written past its end."""
    sets = [make(m, n, B, G, zeros, "f16", xd, seed=i) for i, m in enumerate(ms)]
    x = sets[0][3]
    group = nq.Q4Group([pack(q, s, z, G) for q, s, z, _ in sets])
    need = nq.q4_workspace_bytes(group, B)
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    for yd in (torch.float32, torch.bfloat16):
        bases = [torch.full((B * m + 32,), 7.0, dtype=yd, device=DEV) for m in ms]
        ys = nq.q4_linear_group_into(x.to(DEV), group, [b[16:-16].view(B, m) for b, m in zip(bases, ms)], ws)
        for (q, s, z, _), y, base in zip(sets, ys, bases):
            check(y, x, q, s, z, G)
            assert bool((base[:16] == 7).all()) and bool((base[-16:] == 7).all())
        assert bool((ws[need:] == 0xFF).all())
        # a layer by itself: the same plan or another split, the same bound
        check(nq.q4_linear(x.to(DEV), group.layers[0], out_dtype=yd), x, *sets[0][:3], G)


@pytest.mark.parametrize("m,n,B", [(28672, 8192, 1), (32000, 8192, 4), (8192, 8192, 1)])
def test_large_weights_repeat_their_bits(m, n, B):
    """Weights that are read as a stream, other inputs and another layer in between."""
    layers = [nq.q4_pack(torch.randint(0, 16, (m, n), dtype=torch.uint8, device=DEV),
                         torch.rand(m, n // 128, device=DEV).half(), None, 128) for _ in range(2)]
    xs = [torch.randn(B, n, device=DEV).to(torch.bfloat16) for _ in range(2)]
    first = nq.q4_linear(xs[0], layers[0], out_dtype=torch.float32)
    for k in range(20):
        nq.q4_linear(xs[1], layers[k % 2], out_dtype=torch.float32)
        assert torch.equal(nq.q4_linear(xs[0], layers[0], out_dtype=torch.float32), first)
