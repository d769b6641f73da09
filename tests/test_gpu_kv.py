"""GPU: the paged cache of keys and values: what is written reads back as the oracle's
values bit for bit (each rounding is to the nearest, with ties and quotients as
defined, so there is nothing to tolerate)."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_kv as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ["bf16", "int8", "int4"]
DIMS = [64, 96, 128, 192, 256]


def tokens(rng, T, H, D, dtype):
    x = rng.standard_normal((T, H, D)).astype(np.float32) * np.where(rng.random((1, H, D)) < 0.05, 9, 1)
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def read(cache, slots, dtype=torch.float32):
    return [t.double().cpu().numpy() for t in nq.kv_read(cache, slots, dtype)]


def check(cache, slots, k, v, dtype=torch.float32):
    for got, x in zip(read(cache, slots, dtype), (k, v)):
        want = O.held(x.float().numpy(), cache.kind)
        if dtype == torch.bfloat16:
            want = O.bf16(want.astype(np.float32)).astype(np.float64)
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,H", [(16, 1), (48, 5), (64, 8)])
def test_every_slot(D, kind, dtype, page, H):
    """All slots of three pages, written in a scattered order, read in another."""
    rng = np.random.default_rng([D, page, H])
    cache = nq.KvCache(3, H, D, page=page, kind=kind, device=DEV)
    cache.data.fill_(0xFF)  # NaN or any code
    n = 3 * page
    slots = torch.from_numpy(rng.permutation(n))
    k, v = (tokens(rng, n, H, D, dtype) for _ in range(2))
    nq.kv_write(k.to(DEV), v.to(DEV), cache, slots.to(DEV))
    for out in (torch.float32, torch.bfloat16):
        order = torch.from_numpy(rng.permutation(n))
        check(cache, slots[order].to(DEV), k[order], v[order], out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 17, 65, 300])
def test_token_by_token_leaves_the_others(kind, T):
    """T tokens over an older filling: every other slot keeps its bits, whatever the
    new slots share a tile, a quad of slots or a word with."""
    rng = np.random.default_rng([T, 3])
    H, D, page, pages = 3, 128, 32, 20
    cache = nq.KvCache(pages, H, D, page=page, kind=kind, device=DEV)
    n = pages * page
    k, v = (tokens(rng, n, H, D, torch.float32) for _ in range(2))
    everywhere = torch.arange(n, device=DEV)
    nq.kv_write(k.to(DEV), v.to(DEV), cache, everywhere)
    slots = torch.from_numpy(np.concatenate([np.arange(7, 7 + T // 2), rng.permutation(np.arange(330, n))[:T - T // 2]]))
    nk, nv = (tokens(rng, T, H, D, torch.float32) for _ in range(2))
    nq.kv_write(nk.to(DEV), nv.to(DEV), cache, slots.to(DEV))
    k[slots], v[slots] = nk, nv
    check(cache, everywhere, k, v)


def test_tokens_written_one_call_each_are_those_written_at_once():
    rng = np.random.default_rng(8)
    H, D, T = 2, 64, 37
    k, v = (tokens(rng, T, H, D, torch.bfloat16).to(DEV) for _ in range(2))
    for kind in KINDS:
        a, b = (nq.KvCache(3, H, D, page=16, kind=kind, device=DEV) for _ in range(2))
        a.data.zero_(), b.data.zero_()
        slots = torch.arange(T, device=DEV) + 5
        nq.kv_write(k, v, a, slots)
        for t in range(T):
            nq.kv_write(k[t:t + 1], v[t:t + 1], b, slots[t:t + 1])
        assert torch.equal(a.data, b.data)


@pytest.mark.parametrize("kind", KINDS)
def test_slots_outside_the_cache(kind):
    """Left out when written, zeros when read, up to the ends of 64 bits."""
    rng = np.random.default_rng(9)
    H, D = 2, 96
    cache = nq.KvCache(2, H, D, page=16, kind=kind, device=DEV)
    cache.data.zero_()
    before = cache.data.clone()
    out = torch.tensor([-1, 32, 33, -2 ** 63, 2 ** 63 - 1, 2 ** 32, -2 ** 32 + 3], device=DEV)
    k, v = (tokens(rng, len(out), H, D, torch.float32).to(DEV) for _ in range(2))
    nq.kv_write(k, v, cache, out)
    assert torch.equal(cache.data, before)
    for t in nq.kv_read(cache, out, torch.float32):
        assert not t.any()


@pytest.mark.parametrize("kind", KINDS)
def test_values_at_the_edges(kind):
    """Zeros, the smallest and largest values, ties, infinities and NaN: those stay in
    their head (8 bits) or 32 channels (4 bits)."""
    H, D = 1, 128
    rows = np.zeros((16, H, D), np.float32)
    rows[1] = 1e-45
    rows[2, 0, :64] = 3.4e38
    rows[3, 0] = np.arange(-64, 64)           # ties at every second multiple of the scale
    rows[3, 0, 0] = 127
    rows[4, 0] = np.arange(128) * 0.5 * (7 / 63.5) - 3.5
    rows[5, 0, 3], rows[5, 0, 4:] = np.inf, 1
    rows[6, 0, 40], rows[6, 0, 41:] = np.nan, 2
    rows[7, 0, 100], rows[7, 0, :3] = -np.inf, np.nan
    rows[8] = 2.0 ** -126
    rows[9] = np.linspace(-1e-38, 1e-38, 128)
    rows[10, 0, :] = 1e-30
    rows[10, 0, 5] = 1
    rows[11] = -0.0
    rows[12, 0, ::2], rows[12, 0, 1::2] = 7, 3.5
    rows[13, 0, ::2], rows[13, 0, 1::2] = 127, 0.5
    rows[14] = np.float32(3.4028235e38)
    rows[15, 0, 31], rows[15, 0, 32] = 100, -100
    x = torch.from_numpy(rows)
    cache = nq.KvCache(1, H, D, page=16, kind=kind, device=DEV)
    slots = torch.arange(16, device=DEV)
    nq.kv_write(x.to(DEV), (-x).to(DEV), cache, slots)
    check(cache, slots, x, -x)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_a_wider_output(kind, dtype):
    """k and v as parts of one linear's output, at any element."""
    rng = np.random.default_rng(11)
    T, H, D = 21, 3, 64
    for pad in (0, 1, 3, 8):
        wide = tokens(rng, T, 1, 2 * H * D + 5 + pad, dtype)[:, 0].to(DEV)
        k, v = (wide[:, at:at + H * D].unflatten(1, (H, D)) for at in (pad, pad + H * D + 1))
        cache = nq.KvCache(2, H, D, page=16, kind=kind, device=DEV)
        slots = torch.randperm(32, device=DEV)[:T]
        nq.kv_write(k, v, cache, slots)
        check(cache, slots, k.cpu(), v.cpu())


def test_offsets_beyond_32_bits():
    """A cache of over 4 GiB: the last page is not the one 2^32 bytes before it."""
    rng = np.random.default_rng(12)
    H, D, page = 8, 128, 1024
    cache = nq.KvCache(1060, H, D, page=page, kind="bf16", device=DEV)
    assert cache.data.numel() > 2 ** 32
    slots = torch.tensor([0, 5, 1024 * page + 5, 1059 * page + 1023, 1059 * page], device=DEV)
    k, v = (tokens(rng, 5, H, D, torch.float32) for _ in range(2))
    nq.kv_write(k.to(DEV), v.to(DEV), cache, slots)
    check(cache, slots, k, v)


def test_captured_and_replayed():
    rng = np.random.default_rng(13)
    T, H, D = 9, 2, 128
    for kind in KINDS:
        cache = nq.KvCache(4, H, D, page=16, kind=kind, device=DEV)
        k, v = (tokens(rng, T, H, D, torch.bfloat16).to(DEV) for _ in range(2))
        slots = torch.arange(T, device=DEV)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            nq.kv_write(k, v, cache, slots)
            nq.kv_read(cache, slots)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            nq.kv_write(k, v, cache, slots)
            out = nq.kv_read(cache, slots, torch.float32)
        for i in range(3):
            for t in (k, v):
                t.copy_(tokens(rng, T, H, D, torch.bfloat16))
            slots.copy_(torch.from_numpy(rng.permutation(64)[:T]))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for got, x in zip(out, (k, v)):
                assert np.array_equal(got.double().cpu().numpy(), O.held(x.float().cpu().numpy(), kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts(kind, dtype):
    """Enough tokens that values go four at a time: slots in runs that begin and end
    anywhere, some left out, the last group of four not full."""
    rng = np.random.default_rng(14)
    H, D, page, T = 128, 64, 16, 131
    cache = nq.KvCache(40, H, D, page=page, kind=kind, device=DEV)
    everywhere = torch.arange(40 * page, device=DEV)
    k, v = (tokens(rng, 40 * page, H, D, dtype) for _ in range(2))
    nq.kv_write(k.to(DEV), v.to(DEV), cache, everywhere)
    check(cache, everywhere, k, v)
    runs = [np.arange(4, 45), np.arange(61, 64), np.arange(100, 120), [-1, 300], np.arange(202, 250), np.arange(400, 440)]
    slots = torch.from_numpy(np.concatenate(runs)[:T])
    nk, nv = (tokens(rng, T, H, D, dtype) for _ in range(2))
    nq.kv_write(nk.to(DEV), nv.to(DEV), cache, slots.to(DEV))
    on = slots >= 0
    k[slots[on]], v[slots[on]] = nk[on], nv[on]
    check(cache, everywhere, k, v)
    for got, x in zip(read(cache, slots.to(DEV)), (k, v)):
        assert np.array_equal(got[on.numpy()], O.held(x[slots[on]].float().numpy(), kind)) and not got[~on.numpy()].any()


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_codes_beside_ties(kind):
    """Values on the ties between two codes and next to them on both sides, over scales
    of every size."""
    most = O.MOST[kind]
    D = 256
    group = D if kind == "int8" else 32
    rows = []
    for e in list(range(-126, 121, 13)) + [-130, -133, -99, -100, -101, 99, 100, 101]:
        for scale in (1.0, 1.9921875, 1.3671875):
            s = np.float32(scale) * np.float32(2.0) ** np.float32(e)
            tie = (np.arange(D) % (2 * most) - most + 0.5).astype(np.float32) * s
            for off in (-1, 0, 1):
                x = (tie.view(np.int32) + off).view(np.float32).copy()
                x[::group] = most * s
                rows.append(x)
    x = torch.from_numpy(np.stack(rows)[:, None])
    cache = nq.KvCache(-(-len(rows) // 16), 1, D, page=16, kind=kind, device=DEV)
    slots = torch.arange(len(rows), device=DEV)
    nq.kv_write(x.to(DEV), x.flip(0).to(DEV), cache, slots)
    check(cache, slots, x, x.flip(0))
