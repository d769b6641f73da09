"""GPU: attention of one token over the paged cache, against the fp64 oracle.

Tolerances (derived, not fitted), with e = 2^-24, P = the softmax's weights and
M = sum P |v|.  A score is a sum of D products (of 24 + |c| instead of |c| for 4 bits)
held in fp32: off by under (D + 8) e of the sum of their magnitudes, at most d; a weight
by twice that and 2^-22 for its exponential, and so are the weights' sum and the quotient.
A weight is rounded to bf16, which has 8 significant bits: half a step of 1.0 is 2^-8, and of no value
more; or for fp32 q or y taken as three, off by 2^-23 at most.  The
sum over n tokens is at most n / 32 + 64 sums.  Altogether (2 (2 d + 2^-22) +
w + (n / 32 + 64) e) (M + 24 s for 4 bits), and half a step of the output's type.
Half of the 4-bit products are of 136 + |c| with bf16 q and y, 5.7 times 24, but come 32 to
an instruction: 2 D / 32 + 8 sums, not D + 8, are rounded at that size, 5.7 (D / 16 + 8) / (D + 8)
of what is counted: 0.95 at D = 64, 0.52 at 256."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_kv as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
KINDS = ["bf16", "int8", "int4"]


class Case:
    """Sequences of given lengths over scattered pages of a cache whose other slots, and
    unseen slots of its pages, hold anything."""

    def __init__(self, lengths, Hq=8, H=2, D=128, page=64, kind="bf16", q=BF, y=None, window=0, seed=0, scale=None,
                 loud=1.0, spare=2):
        rng = np.random.default_rng([seed, D, page, Hq, H, len(lengths)])
        self.lengths, self.window, self.kind, self.D, self.H, self.Hq = lengths, window, kind, D, H, Hq
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + spare
        self.cache = nq.KvCache(pages, H, D, page=page, kind=kind, device=DEV)
        self.cache.data.random_(0, 256)
        order = rng.permutation(pages)
        self.table = np.full((len(lengths), max(need + [1])), -7, np.int32)
        at, slots = 0, []
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            t = np.arange(lengths[b])
            slots.append(self.table[b, t // page].astype(np.int64) * page + t % page)
        self.k = [rng.standard_normal((n, H, D)).astype(np.float32) for n in lengths]
        self.v = [rng.standard_normal((n, H, D)).astype(np.float32) + 0.25 for n in lengths]
        self.slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        if len(self.slots):
            nq.kv_write(*(torch.from_numpy(np.concatenate(x)).to(DEV) for x in (self.k, self.v)), self.cache,
                        torch.from_numpy(self.slots).to(DEV))
        self.q = torch.from_numpy((loud * rng.standard_normal((len(lengths), Hq, D))).astype(np.float32)).to(q)
        self.gq, self.gt = self.q.to(DEV), torch.from_numpy(self.table).to(DEV)
        self.gl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        self.y, self.scale = y or q, scale
        # tokens in front of the window may have no page
        if window:
            for b, n in enumerate(lengths):
                self.gt[b, :max(0, n - window) // page] = -1

    def run(self, **kw):
        return nq.kv_attention(self.gq, self.cache, self.gt, self.gl, scale=self.scale, window=self.window,
                               out_dtype=self.y, **kw)

    def check(self, y, rows=None):
        assert y.shape == self.q.shape and y.dtype == self.y
        fine = self.q.dtype == F32 or self.y == F32
        scale = float(np.float32(self.D ** -0.5 if self.scale is None else self.scale))
        got = y.double().cpu().numpy()
        for b in range(len(self.lengths)) if rows is None else rows:
            k, v = O.held(self.k[b], self.kind), O.held(self.v[b], self.kind)
            want, mag, big = O.attention(self.q[b].double().numpy(), k, v, scale, self.window)
            if self.kind == "int4" and len(k):
                s = float(O.scales(self.v[b], "int4").max())
                mag = mag + 24 * s
                sk = float(O.scales(self.k[b], "int4").max())
                big = big + abs(scale) * 24 * sk * np.abs(self.q[b].double().numpy()).sum(1, keepdims=True)
            d = (self.D + 8) * E * big
            w = 2.0 ** -23 if fine else 2.0 ** -8
            n = self.lengths[b]
            tol = (2 * (2 * d + 2.0 ** -22) + w + (n / 32 + 64) * E) * mag
            tol = tol + torch.finfo(self.y).eps / 2 * (np.abs(want) + tol) + 1e-42
            off = np.abs(got[b] - want)
            assert np.all(off <= tol), (b, n, float(np.max(off / tol)))


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 100, 127, 128, 129, 0, 255, 256, 257, 300, 511, 512]


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q,y", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_lengths(D, kind, q, y):
    """One launch (short sequences), and the same lengths beside a longer one."""
    c = Case(LENGTHS, 8, 2, D, 64, kind, q, y)
    c.check(c.run(max_length=512))
    c = Case(LENGTHS + [2100], 8, 2, D, 64, kind, q, y, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (16, 1), (17, 1), (40, 1), (64, 2), (3, 3), (8, 4), (30, 6), (64, 8)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("long", [False, True])
def test_heads(Hq, H, kind, long):
    c = Case([70, 0, 333, 2500 if long else 12], Hq, H, 64, 32, kind, BF, F32)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q", [BF, F32])
def test_more_than_eight_query_heads_a_key_head(D, kind, q):
    for lengths in ([33, 500, 0, 7], [2200, 3, 900]):
        c = Case(lengths, 24, 2, D, 32, kind, q)
        c.check(c.run())


@pytest.mark.parametrize("D", [64, 96, 128, 192])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H", [(17, 1), (64, 2), (99, 3)])
def test_more_than_sixteen_query_heads_a_key_head(D, kind, Hq, H):
    """Some of them 32 at a time: one more than 16, all of 32, one in a second unit; a
    sequence without tokens, cut units and whole ones, a window."""
    c = Case([2600, 0, 40, 1, 700, 33], Hq, H, D, 48, kind, BF)
    c.check(c.run())
    c = Case([1900, 3000], Hq, H, D, 16, kind, BF, window=1700)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q", [BF, F32])
def test_few_and_many_units(D, kind, q):
    """Some tens of units of a few hundred tokens, and several hundred of them: what a
    workgroup has to do with a unit depends on both, and on what is known of the lengths."""
    c = Case([300, 1, 0, 513, 700, 257], 12, 2, D, 32, kind, q)
    for most in (0, 700, 1000, 4000):
        c.check(c.run(max_length=most))
    lengths = [(37 * i) % 301 for i in range(140)]
    c = Case(lengths, 4, 2, D, 32, kind, q)
    c.check(c.run(), list(range(0, 140, 9)))
    c = Case([2000, 1500, 90], 8, 2, D, 32, kind, q, window=400)
    c.check(c.run())


def test_many_sequences():
    """More sequences than a wave has lanes, several times over, most of them empty, in one
    launch and in two."""
    lengths = [(7 * i) % 5 * (i % 3) for i in range(9001)]
    lengths[8000] = 3000
    c = Case(lengths, 2, 1, 64, 16, "int8", BF, F32)
    some = list(range(0, 9001, 97)) + [7999, 8000, 8001, 9000]
    c.check(c.run(), some)
    c.gl[8000] = 17
    c.lengths[8000], c.k[8000], c.v[8000] = 17, c.k[8000][:17], c.v[8000][:17]
    c.check(c.run(max_length=64), some)


@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 1024])
@pytest.mark.parametrize("kind", KINDS)
def test_pages(page, kind):
    for lengths in ([5, 16, 200, 33], [5, 2200, 777, 16]):
        c = Case(lengths, 4, 2, 96, page, kind, F32)
        c.check(c.run())


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 100, 1100, 5000])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
def test_windows(window, kind, page):
    for lengths in ([1, 16, 17, 48, 65, 0, 300], [40, 2500, 1, 1311, 64]):
        c = Case(lengths, 8, 2, 64, page, kind, BF, F32, window=window)
        c.check(c.run())


@pytest.mark.parametrize("lengths", [[40000], [3, 30000, 1, 1, 9000], [1] * 700, [129] * 300, list(range(0, 1200, 7)), list(range(0, 2200, 13))])
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("int8", 128), ("int4", 64)])
def test_shares(lengths, kind, D):
    """One long sequence, a few of very different lengths, many of one token: every way
    that units fall into the workgroups' shares."""
    c = Case(lengths, 4, 2, D, 16, kind, BF, F32)
    if max(lengths) <= 2048:  # a wide table: the host does not know that they are short
        c.gt = torch.cat([c.gt, torch.full((len(lengths), 300), -1, dtype=torch.int32, device=DEV)], dim=1)
    rows = None if len(lengths) < 100 else list(range(0, len(lengths), 17)) + [len(lengths) - 1]
    c.check(c.run(), rows)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("long", [False, True])
def test_loud_scores(kind, long):
    """Scores far apart (one token outweighs the others), falling and rising along the
    sequence, and of one size."""
    for loud in (0.0, 30.0, 1000.0):
        c = Case([400, 37, 2200 if long else 60], 8, 2, 128, 64, kind, F32, loud=loud)
        c.check(c.run())
    c = Case([500, 2400 if long else 250], 2, 1, 64, 16, "bf16", F32)
    for b, up in ((0, 1.0), (1, -1.0)):  # keys that grow along q
        n = c.lengths[b]
        c.k[b][:] = (c.q[b, :1].numpy()[None] * (np.linspace(-3, 3, n) * up)[:, None, None]).astype(np.float32)
    nq.kv_write(*(torch.from_numpy(np.concatenate(x)).to(DEV) for x in (c.k, c.v)), c.cache,
                torch.from_numpy(c.slots).to(DEV))
    c.check(c.run())


def test_scale():
    for scale in (0.0, 1.0, -0.3, 1e-20):
        c = Case([100, 3], 4, 2, 64, 16, "int8", F32, scale=scale)
        c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_what_is_not_seen_does_not_matter(kind):
    """NaN, infinities and any codes in unseen slots, pages and rows: the same bits."""
    for lengths, window in (([1, 17, 100, 250], 0), ([70, 1000, 31], 40), ([70, 2500, 31], 2100)):
        outs = []
        for fill in (0x00, 0xFF, 0x7F, 0x80):
            c = Case(lengths, 8, 2, 128, 32, kind, BF, F32, window=window)
            c.cache.data.fill_(fill)
            seen = np.concatenate([np.arange(n) >= (n - window if window else 0) for n in lengths])
            k, v = (torch.from_numpy(np.concatenate(x)[seen]).to(DEV) for x in (c.k, c.v))
            nq.kv_write(k, v, c.cache, torch.from_numpy(c.slots[seen]).to(DEV))
            outs.append(c.run())
            c.check(outs[-1])
        assert all(torch.equal(outs[0], o) for o in outs)


@pytest.mark.parametrize("long", [False, True])
def test_values_that_are_not_finite(long):
    """As the formula: a NaN key makes its heads NaN, a NaN or infinite value its channel; other
    heads and sequences keep their bits.  8 bits: the whole head; 4 bits: its 32 channels."""
    for kind in KINDS:
        c = Case([60, 61, 2200 if long else 62], 4, 2, 64, 16, kind, BF, F32)
        clean = c.run()
        first = torch.from_numpy(c.slots[:1]).to(DEV)
        k, v = torch.from_numpy(c.k[0][:1]).to(DEV), torch.from_numpy(c.v[0][:1]).to(DEV)
        v[0, 0, 5], k[0, 1, 3] = float("nan"), float("nan")
        nq.kv_write(k, v, c.cache, first)
        y = c.run()
        assert torch.equal(y[1:], clean[1:])
        assert torch.isnan(y[0, 2:]).all()
        cut = {"bf16": slice(5, 6), "int8": slice(0, 64), "int4": slice(0, 32)}[kind]
        hit = torch.zeros(64, dtype=torch.bool)
        hit[cut] = True
        assert torch.isnan(y[0, :2][:, hit]).all() and torch.equal(y[0, :2][:, ~hit], clean[0, :2][:, ~hit])


def test_queries_that_are_not_finite_stay_in_their_head():
    for q in (BF, F32):
        for long in (False, True):
            c = Case([50, 2300 if long else 70], 8, 2, 64, 16, "int4", q)
            clean = c.run()
            c.gq[0, 3, 7], c.gq[1, 6, 0] = float("nan"), float("inf")
            y = c.run()
            hit = torch.zeros(2, 8, dtype=torch.bool)
            hit[0, 3] = hit[1, 6] = True
            assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("q", [BF, F32])
@pytest.mark.parametrize("long", [False, True])
def test_scores_that_are_all_minus_infinity(long, q):
    """Nothing to weigh is no number, as the formula has it, and not zeros; one finite score
    takes all the weight.  Products with 2 of q's -3e38 pass the largest value of fp32, and with
    127 of 8 bits; 4 bits take 7 / 16 of it for fp32 q (-1.3e38, and the scores times
    scale stay finite): the formula's values, tied tokens alike."""
    for kind in KINDS:
        c = Case([40, 2300 if long else 70], 4, 2, 64, 16, kind, q)
        first = torch.from_numpy(c.slots).to(DEV)
        k, v = torch.from_numpy(np.concatenate(c.k)).to(DEV), torch.from_numpy(np.concatenate(c.v)).to(DEV)
        k[..., 3] = 2.0
        k[5, 0, 3] = k[45, 1, 3] = 0.0
        nq.kv_write(k, v, c.cache, first)
        clean = c.run()
        c.gq[0, :, 3] = c.gq[1, :, 3] = -3e38
        y = c.run()
        assert torch.isfinite(clean).all()
        if kind == "int4" and q == F32:
            for b, at in ((0, slice(0, 40)), (1, slice(40, None))):
                held = [O.held(t[at].cpu().numpy(), kind) for t in (k, v)]
                want, mag, _ = O.attention(c.gq[b].double().cpu().numpy(), *held, 64 ** -0.5)
                # equal weights of one: n sums, their quotient and the scales' products, 2^-24 each
                assert np.all(np.abs(y[b].double().cpu().numpy() - want) <= (c.lengths[b] / 32 + 72) * E * mag)
            continue
        assert torch.isnan(y[0, 2:]).all() and torch.isnan(y[1, :2]).all()
        if kind == "bf16":
            assert torch.equal(y[0, :2], v[5, 0].bfloat16().to(q).expand(2, -1))
            assert torch.equal(y[1, 2:], v[45, 1].bfloat16().to(q).expand(2, -1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("long", [False, True])
def test_bad_lengths_and_pages_make_their_sequence_nan(kind, long):
    """Lengths below zero or above what the table or max_length allow, pages outside the
    cache: NaN for that sequence, its neighbours keep their bits."""
    n = 2500 if long else 130
    c = Case([n, 100, 64, 33, 90, 20], 4, 2, 64, 16, kind, BF, F32)
    want = c.run()
    bad = c.gl.clone()
    bad[1], bad[3] = -5, c.gt.shape[1] * 16 + 1
    c.gt[4, 2] = c.cache.pages
    c.gt[5, 0] = -1
    c.gl = bad
    y = c.run()
    assert torch.isnan(y[[1, 3, 4, 5]]).all()
    assert torch.equal(y[[0, 2]], want[[0, 2]])
    if not long:
        assert torch.isnan(c.run(max_length=90)[0]).all()


def test_repeated_and_reordered_batches():
    """Repeated calls give the same bits; in one launch a sequence's bits do not depend on
    the batch either."""
    c = Case([100, 0, 512, 77, 300], 8, 2, 128, 64, "int8")
    a = c.run(max_length=512)
    assert torch.equal(a, c.run(max_length=512))
    some = torch.tensor([3, 2, 0], device=DEV)
    y = nq.kv_attention(c.gq[some], c.cache, c.gt[some], c.gl[some], max_length=512)
    assert torch.equal(y, a[some])
    c = Case([9000, 1, 2500, 31], 8, 2, 128, 64, "int8")
    assert torch.equal(c.run(), c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed_while_sequences_grow(kind):
    """One captured call over lengths and a table that change between the replays, on a
    workspace that eager calls use in between."""
    c = Case([700, 40, 0, 2300], 8, 2, 128, 16, kind, BF)
    ws = nq.new_kv_workspace(4, 8, c.cache)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = c.run(workspace=ws)
    for lengths in ([700, 40, 0, 2300], [1, 17, 0, 600], [640, 0, 0, 1], [0, 0, 0, 0], [699, 33, 0, 1299]):
        c.gl.copy_(torch.tensor(lengths, dtype=torch.int32))
        c.gq.copy_(torch.randn(c.gq.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(sum(lengths))))
        want = c.run(workspace=ws)
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_two_streams_at_once():
    cases = [Case([5000, 3, 900], 8, 2, 128, 64, "bf16", seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            got.append(c.run(stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_beyond_32_bits():
    """Pages on both sides of 2^32 bytes of one cache."""
    rng = np.random.default_rng(12)
    H, D, page = 8, 128, 1024
    cache = nq.KvCache(1060, H, D, page=page, kind="bf16", device=DEV)
    table = torch.tensor([[1059, 3], [35, 1058]], dtype=torch.int32, device=DEV)
    c = Case.__new__(Case)
    c.lengths, c.window, c.kind, c.D, c.H, c.Hq, c.scale, c.y = [1500, 1030], 0, "bf16", D, H, 16, None, F32
    c.k = [rng.standard_normal((n, H, D)).astype(np.float32) for n in c.lengths]
    c.v = [rng.standard_normal((n, H, D)).astype(np.float32) for n in c.lengths]
    slots = np.concatenate([table.cpu().numpy()[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
                            for b, n in enumerate(c.lengths)])
    nq.kv_write(*(torch.from_numpy(np.concatenate(x)).to(DEV) for x in (c.k, c.v)), cache, torch.from_numpy(slots).to(DEV))
    c.q = torch.from_numpy(rng.standard_normal((2, 16, D)).astype(np.float32))
    c.check(nq.kv_attention(c.q.to(DEV), cache, table, torch.tensor(c.lengths, dtype=torch.int32, device=DEV)))
