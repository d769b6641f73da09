"""GPU: 4-bit linears whose activations and scales lie far apart, so that their
product is an ordinary number and a step on the way to it need not be.

Tolerance: that of the other parity tests of these linears.  Their bound holds one
sum for each group at 2^-23 of M, twice an fp32 rounding; what is rounded besides
is s times a group's sum, by 2^-24 of that group's part of M."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_q4 as Q
from tests.test_gpu_q4 import DEV, DT, check, f64, make, pack

pytestmark = pytest.mark.gpu

# shared and split decode, both prompt tiles, K splits
SHAPES = [(70, 300, 1), (70, 300, 16), (130, 9000, 7), (64, 28672, 16), (70, 300, 17), (40, 1100, 64), (70, 300, 65),
          (130, 2179, 130)]


def far(m, n, B, G, scale, xd, s_power, x_power):
    q, s, z, x = make(m, n, B, G, True, scale, xd)
    s = (s.double() * 2.0 ** s_power).to(DT[scale])
    return q, s, z, (x.double() * 2.0 ** x_power).to(DT[xd])


@pytest.mark.parametrize("m,n,B", SHAPES)
@pytest.mark.parametrize("G", [32, 128])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("scale,s_power", [("f16", -10), ("f32", -20), ("f32", -60)])
@pytest.mark.parametrize("x_power", [113, 120])
def test_large_activations_and_small_scales(m, n, B, G, xd, scale, s_power, x_power):
    """Outputs of about 2^120 at most; a group's sum without its scale passes fp32."""
    q, s, z, x = far(m, n, B, G, scale, xd, s_power, x_power)
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, G), out_dtype=torch.float32), x, q, s, z, G)


@pytest.mark.parametrize("m,n,B", SHAPES)
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("scale", ["f16", "f32"])
def test_zero_scales_and_large_activations(m, n, B, xd, scale):
    """A group whose scale is zero adds nothing, whatever its sum."""
    q, s, z, x = far(m, n, B, 64, scale, xd, 0, 0)
    block = slice(128, 256)  # whole, for columns beside them would share their power of two
    x[:, block] = (x[:, block].double() * 2.0 ** 123).to(DT[xd])
    s[:, 2:4] = 0
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32)
    assert bool(torch.isfinite(y).all())
    if B <= 16:  # above, the power of two is the row's
        x[:, block] = 0
        check(y, x, q, s, z, 64)


@pytest.mark.parametrize("m,n,B", SHAPES)
@pytest.mark.parametrize("G", [32, 128])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_small_activations_and_large_scales(m, n, B, G, xd):
    q, s, z, x = far(m, n, B, G, "f32", xd, 75, -90)
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, G), out_dtype=torch.float32), x, q, s, z, G)


# ------------------------------------------------------------------ scales at pack time
@pytest.mark.parametrize("B", [1, 17, 130])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_scale_that_is_taken(B, sign):
    """Every scale just below 2^80, and activations that make the outputs ordinary: no
    sum on the way passes fp32 in either kernel."""
    q, s, z, x = far(40, 300, B, 32, "f32", "f32", 0, -90)
    s = torch.full_like(s, sign * 2.0 ** 80 * (1 - 2.0 ** -24))
    check(nq.q4_linear(x.to(DEV), pack(q, s, z, 32), out_dtype=torch.float32), x, q, s, z, 32)


@pytest.mark.parametrize("value", [2.0 ** 80, -2.0 ** 80, 2.0 ** 110, -3.4e38])
@pytest.mark.parametrize("zeros", [True, False])
def test_larger_scales_are_refused(value, zeros):
    """From 2^102 on, a prompt's sum of scale times integers passes fp32 before the
    power of two of a small x is applied, where the same call for 16 rows was right."""
    q, s, z, _ = make(40, 300, 1, 64, zeros, "f32", "f32")
    s[39, 4] = value
    with pytest.raises(nq.NQError) as e:
        pack(q, s, z, 64)
    assert e.value.status == nq.NQ_ERR_RANGE and "scale" in str(e.value)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("scale", ["f16", "f32"])
@pytest.mark.parametrize("B", [2, 30])
def test_infinite_and_nan_scales_stay_in_their_row(value, scale, B):
    q, s, z, x = make(40, 300, B, 64, True, scale, "bf16")
    ref = nq.q4_linear(x.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32)
    s[21, 4] = value
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, 64), out_dtype=torch.float32)
    assert not torch.isfinite(y[:, 21]).any()
    keep = [i for i in range(40) if i != 21]
    assert torch.equal(y[:, keep], ref[:, keep])


# ------------------------------------------------------------------ the smallest activations
@pytest.mark.parametrize("B", [1, 16, 17, 130])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("x_power", [-115, -128, -138])
def test_activations_below_the_normal_numbers(B, xd, x_power):
    """Besides the usual bound, half a step of 2^-144 for each fp32 x; a bf16 x is a
    multiple of 2^-133 and loses nothing."""
    m, n, G = 70, 300, 64
    q, s, z, x = far(m, n, B, G, "f32", xd, 75, x_power)
    y = nq.q4_linear(x.to(DEV), pack(q, s, z, G), out_dtype=torch.float32)
    ref, M = Q.linear(f64(x), q, f64(s), z, G), Q.magnitude(f64(x), q, f64(s), z, G)
    chain = 128 * (2 if xd == "f32" else 1) + -(-n // G) + 32
    tol = (chain * 2.0 ** -23 + 2.0 ** -22) * M
    tol = tol + 2.0 ** -39 * np.abs(f64(x)).max(1, keepdims=True) * np.abs(Q.weight(q, f64(s), z, G)).sum(1)
    if xd == "f32":
        tol = tol + 2.0 ** -145 * np.abs(Q.weight(q, f64(s), z, G)).sum(1)
    assert np.all(np.abs(f64(y) - ref) <= tol)
