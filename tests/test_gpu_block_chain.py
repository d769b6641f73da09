"""GPU: a block of a compressed model as it is decoded: norms, binary linears and
4-bit linears one after another, eager, captured and replayed, and on two
streams at once."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
import synth
from oracle import nq_norm, nq_oracle, nq_q4
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DEV = G.DEV
D, WIDE, VOCAB = 512, 1100, 1000
f64 = lambda t: t.double().cpu().numpy()


class Chain:
    """norm, 4-bit q/k/v, binary o, norm, binary gate/up, 4-bit down, norm, 4-bit head."""

    def __init__(self, B, seed=0):
        rng = np.random.default_rng([seed, B])
        self.B = B

        def four(m, n):
            q = rng.integers(0, 16, (m, n)).astype(np.uint8)
            s = (rng.random((m, -(-n // 64))).astype(np.float32) * 0.2 / np.sqrt(n)).astype(np.float16)
            z = rng.integers(4, 12, s.shape).astype(np.uint8)
            return (q, s, z), nq.q4_pack(*(torch.from_numpy(t).to(DEV) for t in (q, s, z)), group=64)

        def binary(m, n, r, layer):
            L = synth.make_layer(m, n, r, 1, cfg=60, layer=layer)
            L.s1 = (L.s1.astype(np.float32) / (n * r) ** 0.5).astype(np.float16)
            return L, G.pack_layer(L)
        self.qkv = [four(m, D) for m in (D, 128, 128)]
        self.group = nq.Q4Group([p for _, p in self.qkv])
        self.o = binary(D, D, 300, 0)
        self.gate_up = [binary(WIDE, D, 260, i) for i in (1, 2)]
        self.down, self.head = four(D, WIDE), four(VOCAB, D)
        self.w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(D).astype(np.float32)).to(DEV) for _ in range(2)]
        self.norm = nq.BlockNorm(D, res_dtype=torch.float32, w_post=self.w[0], w_pre=self.w[1], res_scale=0.9)
        self.h = torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)).to(DEV)

    def run(self, h):
        """(logits, h', and every step's (kind, inputs, outputs))."""
        seen = []
        s, x = nq.block_norm(h, None, self.norm)
        seen.append(("pre", (h,), (x,)))
        q = nq.q4_linear_group(x, self.group)
        seen.append(("qkv", (x,), q))
        y = nq.linear(q[0], self.o[1])
        seen.append(("o", (q[0],), (y,)))
        s2, x = nq.block_norm(s, y, self.norm)
        seen.append(("norm", (s, y), (s2, x)))
        g = nq.linear_group(x, [p for _, p in self.gate_up])
        seen.append(("gate_up", (x,), g))
        y = nq.q4_linear(g[0] * g[1], self.down[1])
        seen.append(("down", (g[0] * g[1],), (y,)))
        s3, x = nq.block_norm(s2, y, self.norm)
        seen.append(("norm", (s2, y), (s3, x)))
        logits = nq.q4_linear(x, self.head[1], out_dtype=torch.float32)
        seen.append(("head", (x,), (logits,)))
        return logits, s3, seen

    def reference(self, kind, ins):
        """The step's outputs from its inputs, in fp64."""
        wp, wq = f64(self.w[0]), f64(self.w[1])
        q4 = lambda x, t: nq_q4.linear(f64(x), *t, 64)
        bits = lambda x, L: nq_oracle.linear_factored(f64(x), L.U, L.V, *(v.astype(np.float64) for v in (L.s1, L.g, L.s2)))
        a, eps = float(np.float32(0.9)), float(np.float32(1e-5))
        if kind == "pre":
            return [nq_norm.forward(f64(ins[0]), None, wp, wq, None, a, 1.0, eps)[1]]
        if kind == "norm":
            return nq_norm.forward(f64(ins[0]), f64(ins[1]), wp, wq, None, a, 1.0, eps)
        if kind == "qkv":
            return [q4(ins[0], t) for t, _ in self.qkv]
        if kind == "gate_up":
            return [bits(ins[0], L) for L, _ in self.gate_up]
        if kind == "o":
            return [bits(ins[0], self.o[0])]
        return [q4(ins[0], (self.down if kind == "down" else self.head)[0])]


@pytest.mark.parametrize("B", [1, 3, 16, 40, 130])
def test_every_step_of_the_chain(B):
    """Relative L2 of each step from its own inputs: half a step of a bf16 output
    (2^-8 at most) and, for the binary linears, their 2e-3."""
    c = Chain(B)
    for kind, ins, outs in c.run(c.h)[2]:
        for got, ref in zip(outs, c.reference(kind, ins)):
            bar = (2.0 ** -8 if got.dtype == torch.bfloat16 else 2e-6) + (2e-3 if kind in ("o", "gate_up") else 0)
            assert G.rel_l2(f64(got), ref) <= bar, (kind, G.rel_l2(f64(got), ref))


@pytest.mark.parametrize("B", [1, 16, 130])
def test_captured_and_replayed(B):
    """Every replay gives the bits of the eager run on the same stream of inputs,
    with eager work and synchronisations in between."""
    c = Chain(B)
    h = c.h.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        logits, out, _ = c.run(h)
    for k in range(4):
        h.copy_(torch.randn(B, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(k)) * (k + 1))
        want, want_h, _ = c.run(h)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logits, want) and torch.equal(out, want_h)


@pytest.mark.parametrize("B", [1, 130])
def test_gradients_captured_and_replayed(B):
    norm = nq.BlockNorm(D, act_dtype=torch.float32, w_post=torch.rand(D, device=DEV), w_pre=torch.rand(D, device=DEV),
                        gate=torch.rand(D, device=DEV))
    gen = torch.Generator(device=DEV).manual_seed(3)
    t = [torch.randn(B, D, device=DEV, generator=gen) for _ in range(4)]

    def run():
        h, x, stats = nq.block_norm(t[0], t[1], norm, with_stats=True)
        return {"h": h, "x": x, **nq.block_norm_backward(t[2], t[3], h, t[1], stats, norm)}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = run()
    for k in range(4):
        for v in t:
            v.copy_(torch.randn(B, D, device=DEV, generator=gen))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(kept[name], want[name]), name


def test_two_streams_at_once():
    """The chain on two streams, each with buffers and workspaces of its own."""
    chains = [Chain(130, seed=s) for s in (1, 2)]
    want = [c.run(c.h)[0] for c in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(3):
        got = []
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                got.append(c.run(c.h)[0])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_training_step_through_a_binary_linear():
    """x = norm(h), y = W x on a binary linear, dx = W^T dy on its transposed layer,
    then the norm's gradients: the slope of sum(y dy) along a direction of h, by
    differences of the fp64 oracle at the same point."""
    L = synth.make_layer(300, D, 200, 4, cfg=61)
    layer = G.pack_layer(L)
    w = torch.rand(D, device=DEV) + 0.5
    norm = nq.BlockNorm(D, act_dtype=torch.float32, w_pre=w)
    h = torch.randn(4, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    _, x, stats = nq.block_norm(h, None, norm, with_stats=True)
    dy = torch.randn(4, 300, device=DEV, generator=torch.Generator(device=DEV).manual_seed(6))
    dx = nq.linear(dy, nq.transpose(layer))
    dh = nq.block_norm_backward(dx, None, h, None, stats, norm)["dh"]

    def loss(hh):
        xx = nq_norm.forward(hh, None, None, f64(w), None, 1.0, 1.0, float(np.float32(1e-5)))[1]
        y = nq_oracle.linear_factored(xx, L.U, L.V, *(v.astype(np.float64) for v in (L.s1, L.g, L.s2)))
        return float(np.sum(y * f64(dy)))
    rng = np.random.default_rng(7)
    way = rng.standard_normal((4, D))
    slope = (loss(f64(h) + 1e-5 * way) - loss(f64(h) - 1e-5 * way)) / 2e-5
    # the transposed product is within 3e-4 (relative L2); the differences within 1e-6
    assert abs(slope - float(np.sum(f64(dh) * way))) <= 1e-3 * np.linalg.norm(f64(dh)) * np.linalg.norm(way)
