"""GPU: the attention half of a block as it is decoded: norm, 4-bit q/k/v, norm and
rotation of the heads into the cache, attention over the cache, binary output linear; a
prompt first, then token after token, eager, captured and replayed while the
sequences grow, and on two streams at once."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
import synth
from oracle import nq_heads, nq_kv, nq_norm, nq_oracle, nq_q4
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DEV = G.DEV
D, HQ, HK, HD, PAGE = 512, 8, 2, 64, 16
f64 = lambda t: t.double().cpu().numpy()


class Block:
    """B sequences with room for `room` tokens each, pages scattered over the cache."""

    def __init__(self, B, kind, room, seed=0):
        rng = np.random.default_rng([seed, B])
        self.B, self.kind = B, kind

        def four(m, n):
            q = rng.integers(0, 16, (m, n)).astype(np.uint8)
            s = (rng.random((m, -(-n // 64))).astype(np.float32) * 0.3 / np.sqrt(n)).astype(np.float16)
            return (q, s, None), nq.q4_pack(*(torch.from_numpy(t).to(DEV) for t in (q, s)), group=64)
        self.qkv = [four(m, D) for m in (HQ * HD, HK * HD, HK * HD)]
        self.group = nq.Q4Group([p for _, p in self.qkv])
        L = synth.make_layer(D, HQ * HD, 300, 1, cfg=70)
        L.s1 = (L.s1.astype(np.float32) / (300 * HQ * HD) ** 0.5).astype(np.float16)
        self.o, self.o_packed = L, G.pack_layer(L)
        self.w_pre = torch.from_numpy(1 + 0.2 * rng.standard_normal(D).astype(np.float32)).to(DEV)
        self.norm = nq.BlockNorm(D, w_pre=self.w_pre, post=False)
        self.w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(HD).astype(np.float32)).to(DEV) for _ in range(2)]
        self.freq = 10000.0 ** (-np.arange(0, HD, 2) / HD)
        self.heads = nq.HeadNorm(HD, w_q=self.w[0], w_k=self.w[1], inv_freq=torch.from_numpy(self.freq).to(DEV))
        pages = -(-room // PAGE)
        self.cache = nq.KvCache(B * pages + 1, HK, HD, page=PAGE, kind=kind, device=DEV)
        self.table = torch.from_numpy(rng.permutation(B * pages).astype(np.int32).reshape(B, pages)).to(DEV)
        self.ws = nq.new_kv_workspace(B, HQ, self.cache)
        self.rng = rng

    def inputs(self, rows):
        return torch.from_numpy(self.rng.standard_normal((rows, D)).astype(np.float32)).to(DEV).bfloat16()

    def slots(self, b, at):
        return self.table[b].long()[at // PAGE] * PAGE + at % PAGE

    def linears(self, h):
        x = nq.block_norm(h, None, self.norm)[1]
        q, k, v = nq.q4_linear_group(x, self.group)
        return x, *(t.unflatten(1, (-1, HD)) for t in (q, k, v))

    def prompt(self, b, n):
        """The first n tokens of sequence b."""
        h, at = self.inputs(n), torch.arange(n, device=DEV)
        _, q, k, v = self.linears(h)
        _, k2 = nq.head_norm(q, k, at, self.heads)
        nq.kv_write(k2, v, self.cache, self.slots(b, at))

    def step(self, h, lengths):
        """One new token a sequence, lengths (device) with it; every step's in- and outputs."""
        last = lengths.long() - 1
        slots = (self.table.long().gather(1, (last // PAGE)[:, None])[:, 0] * PAGE + last % PAGE)
        x, q, k, v = self.linears(h)
        q2 = nq.head_norm_write(q, k, v, last, self.heads, self.cache, slots)
        a = nq.kv_attention(q2, self.cache, self.table, lengths, workspace=self.ws)
        y = nq.linear(a.flatten(1), self.o_packed)
        return {"x": x, "q": q, "k": k, "v": v, "q2": q2, "a": a, "y": y, "slots": slots}

    def check(self, h, lengths, s):
        """Relative L2 of each step from its own inputs: half a step of a bf16 output (2^-8
        at most), as much again for the softmax's weights, and the binary linear's 2e-3."""
        half = 2.0 ** -8
        want = nq_norm.forward(f64(h), None, None, f64(self.w_pre), None, 1.0, 1.0, float(np.float32(1e-5)))[1]
        assert G.rel_l2(f64(s["x"]), want) <= half
        for name, (t, _) in zip("qkv", self.qkv):
            assert G.rel_l2(f64(s[name].flatten(1)), nq_q4.linear(f64(s["x"]), *t, 64)) <= half
        n = lengths.cpu().numpy()
        phi = nq_heads.angles((n - 1)[None], self.freq, (HD // 2,))
        eps = float(np.float32(1e-6))
        q2, k2 = (nq_heads.forward(f64(s[m]), f64(w), phi, False, eps)[0] for m, w in zip("qk", self.w))
        assert G.rel_l2(f64(s["q2"]), q2) <= half
        kept = nq.kv_read(self.cache, s["slots"], torch.float32)
        # a key may be the other neighbour in bf16 (2^-7 of it) before it becomes a code
        room = {"bf16": 0.0, "int8": 1 / 127, "int4": 1 / 7}[self.kind]
        top = np.abs(k2).max(axis=-1, keepdims=True)
        assert np.all(np.abs(f64(kept[0]) - k2) <= (2.0 ** -7 + 2.0 ** -8) * np.abs(k2) + room * top)
        assert np.array_equal(f64(kept[1]), nq_kv.held(s["v"].float().cpu().numpy(), self.kind))
        for b in range(self.B):
            at = torch.arange(int(n[b]), device=DEV)
            k, v = nq.kv_read(self.cache, self.slots(b, at), torch.float32)
            ref, _, _ = nq_kv.attention(f64(s["q2"][b]), f64(k), f64(v), HD ** -0.5)
            assert G.rel_l2(f64(s["a"][b]), ref) <= 2 * half
        L = self.o
        bits = nq_oracle.linear_factored(f64(s["a"].flatten(1)), L.U, L.V, *(v.astype(np.float64) for v in (L.s1, L.g, L.s2)))
        assert G.rel_l2(f64(s["y"]), bits) <= 2e-3 + half


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("room", [200, 3000])
def test_prompt_then_tokens(kind, room):
    """Prompts of different lengths (one sequence without any), then five tokens."""
    c = Block(4, kind, room)
    prompts = [room - 20, 0, 33, 95]
    for b, n in enumerate(prompts):
        c.prompt(b, n)
    lengths = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    for _ in range(5):
        lengths += 1
        h = c.inputs(4)
        c.check(h, lengths, c.step(h, lengths))


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("room", [200, 3000])
def test_captured_and_replayed_token_after_token(kind, room):
    """One captured step for every token: each replay gives the bits of an eager step on the
    same cache, with eager work and synchronisations in between."""
    c = Block(3, kind, room)
    for b, n in enumerate((room - 30, 10, 64)):
        c.prompt(b, n)
    start = torch.tensor([room - 30, 10, 64], dtype=torch.int32, device=DEV)
    lengths, h = start + 1, c.inputs(3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.step(h, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = c.step(h, lengths)
    for k in range(4):
        lengths.copy_(start + 1 + k)
        h.copy_(c.inputs(3))
        want = c.step(h, lengths)
        data = c.cache.data.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(kept[n], want[n]) for n in want) and torch.equal(c.cache.data, data)


def test_two_streams_at_once():
    blocks = [Block(3, kind, 1500, seed=s) for s, kind in enumerate(("int8", "bf16"))]
    lengths = torch.tensor([1400, 77, 300], dtype=torch.int32, device=DEV)
    hs = [c.inputs(3) for c in blocks]
    for c in blocks:
        for b, n in enumerate((1399, 76, 299)):
            c.prompt(b, n)
    want = [c.step(h, lengths)["y"] for c, h in zip(blocks, hs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        got = []
        for c, h, s in zip(blocks, hs, streams):
            with torch.cuda.stream(s):
                got.append(c.step(h, lengths)["y"])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_training_step_through_the_heads():
    """q = norm and rotation of W x on a binary linear, backward through both: the slope of
    sum(q g) along a direction of x, by differences of the fp64 oracle."""
    L = synth.make_layer(4 * HD, D, 200, 4, cfg=71)
    layer, T = G.pack_layer(L), 6
    w = torch.rand(HD, device=DEV) + 0.5
    freq = 100.0 ** (-np.arange(0, HD, 2) / HD)
    norm = nq.HeadNorm(HD, act_dtype=torch.float32, w_q=w, inv_freq=torch.from_numpy(freq).to(DEV))
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, g = torch.randn(T, D, device=DEV, generator=gen), torch.randn(T, 4, HD, device=DEV, generator=gen)
    at = torch.arange(T, device=DEV)
    y = nq.linear(x, layer).unflatten(1, (4, HD))
    dq = nq.head_norm_backward(g, None, y, None, at, norm)["dq"]
    dx = nq.linear(dq.flatten(1), nq.transpose(layer))
    phi = nq_heads.angles(at.cpu().numpy()[None], freq, (HD // 2,))

    def loss(xx):
        yy = nq_oracle.linear_factored(xx, L.U, L.V, *(v.astype(np.float64) for v in (L.s1, L.g, L.s2)))
        q = nq_heads.forward(yy.reshape(T, 4, HD), f64(w), phi, False, float(np.float32(1e-6)))[0]
        return float(np.sum(q * f64(g)))
    way = np.random.default_rng(7).standard_normal((T, D))
    slope = (loss(f64(x) + 1e-5 * way) - loss(f64(x) - 1e-5 * way)) / 2e-5
    # both products are within 3e-4 (relative L2), the differences within 1e-6
    assert abs(slope - float(np.sum(f64(dx) * way))) <= 2e-3 * np.linalg.norm(f64(dx)) * np.linalg.norm(way)
