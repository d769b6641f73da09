"""GPU: 4-bit linears and block norms on tensors whose elements or bytes pass 2^32:
the last rows have the bits of a call on those rows alone."""
import pytest
import torch

import binary_rank_gemv_packed_amd as nq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LAST = 130


@pytest.fixture(autouse=True)
def give_back():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def test_norm_rows_beyond_32_bits():
    rows, d = 280000, 16384  # 4.6e9 values
    w = torch.rand(d, device=DEV)
    norm = nq.BlockNorm(d, w_post=w, w_pre=w, gate=w)
    gen = torch.Generator(device=DEV).manual_seed(1)
    h, y = (torch.empty(rows, d, dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for _ in range(2))
    h_out, x, stats = nq.block_norm(h, y, norm, with_stats=True)
    ends = [t[-LAST:].clone() for t in (h, y)]
    ho, xo, st = nq.block_norm(*ends, norm, with_stats=True)
    assert torch.equal(h_out[-LAST:], ho) and torch.equal(x[-LAST:], xo) and torch.equal(stats[:, -LAST:], st)
    got = nq.block_norm_backward(x, h, h_out, y, stats, norm)
    end = nq.block_norm_backward(xo, ends[0], ho, ends[1], st, norm)
    for k in ("dh", "dy"):
        assert torch.equal(got[k][-LAST:], end[k]), k
    # dw_pre = sum of w hn^2, terms of one sign: each of the three sums is off by at most
    # 2^-24 of itself for each of 1094 rows of a workgroup and 272 additions of the join
    rest = nq.block_norm_backward(x[:-LAST], h[:-LAST], h_out[:-LAST], y[:-LAST], stats[:, :-LAST].contiguous(), norm)
    off = (got["dw_pre"] - rest["dw_pre"] - end["dw_pre"]).abs()
    assert bool((off <= 2 * (1094 + 272 + 2) * 2.0 ** -24 * got["dw_pre"]).all())


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_prompt_outputs_beyond_32_bits(xd):
    m, n, B = 65536, 100, 70000  # 4.6e9 outputs
    layer = nq.q4_pack(torch.randint(0, 16, (m, n), dtype=torch.uint8, device=DEV), torch.rand(m, 1, device=DEV).half())
    x = torch.randn(B, n, device=DEV).to(xd)
    y = nq.q4_linear(x, layer, out_dtype=torch.bfloat16)
    assert torch.equal(y[-LAST:], nq.q4_linear(x[-LAST:].contiguous(), layer, out_dtype=torch.bfloat16))


def test_prompt_activations_beyond_32_bits():
    m, n, B = 64, 65536, 70000  # 4.6e9 activations, 9.2 GB of them in fp16 beside
    layer = nq.q4_pack(torch.randint(0, 16, (m, n), dtype=torch.uint8, device=DEV), torch.rand(m, n // 128, device=DEV).half())
    x = torch.empty(B, n, dtype=torch.bfloat16, device=DEV).normal_()
    y = nq.q4_linear(x, layer, out_dtype=torch.float32)
    end = nq.q4_linear(x[-LAST:].contiguous(), layer, out_dtype=torch.float32)
    # fewer rows are split over the columns: sums in another order
    assert float((y[-LAST:] - end).norm() / end.norm()) <= 1e-5


@pytest.mark.parametrize("B", [1, 16, 20])
def test_codes_beyond_32_bits(B):
    m, n = 1 << 20, 8320  # 4.4e9 bytes of codes
    codes = torch.randint(0, 16, (m, n), dtype=torch.uint8, device=DEV)
    scales = torch.rand(m, n // 64, device=DEV).half()
    zeros = torch.randint(0, 16, scales.shape, dtype=torch.uint8, device=DEV)
    layer = nq.q4_pack(codes, scales, zeros, 64)
    x = torch.randn(B, n, device=DEV).to(torch.bfloat16)
    y = nq.q4_linear(x, layer, out_dtype=torch.float32)
    end = slice(m - 4096, m)
    part = nq.q4_pack(codes[end], scales[end], zeros[end], 64)
    want = nq.q4_linear(x, part, out_dtype=torch.float32)
    if B > 1:  # fewer rows of W are split over the columns: sums in another order
        assert float((y[:, end] - want).norm() / want.norm()) <= 1e-5
    else:
        assert torch.equal(y[:, end], want)
    back, z = nq.q4_unpack(layer)
    assert torch.equal(back[end], codes[end]) and torch.equal(z[end], zeros[end])
