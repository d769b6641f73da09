"""GPU: norms and rotation of heads and their gradients against the fp64 oracle.

Tolerances (derived, not fitted), with e = 2^-24.  A sum of D squares is at most 8
sums in a lane and 6 over lanes, so 1/rms is off by under (14 + 3) / 2 e + 2 e, and x r w
by under 14 e of itself.  The angle's fraction of a turn is rounded to fp32 (pi 2^-25 of
a sine at most), sine and cosine are off by 4 e at most; products and their sum
by 2 e more: F = 24 e of the magnitudes |n_a| + |n_b|.  Backward: g is off by 8 e of
|dy_a| + |dy_b|, each mean by 16 e of the mean of magnitudes, the rest as in the
forward: G = 64 e of the formula's magnitudes; a sum over T tokens of H heads by
another (T H + 64) e at most.  An output is rounded once, by half a step of its type.
An angle of phi radians is formed to 2^-52 phi: below 2^24 radians that is under e."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_heads as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
F, GRAD = 24, 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, T, Hq, Hk, D, rot=None, interleaved=False, sections=None, act="f32", par="f32", norm=True,
                 weights=True, offset=0.0, far=5000, seed=0, eps=1e-6):
        rng = np.random.default_rng([seed, T, Hq, Hk, D])
        rot = D if rot is None else rot
        t = lambda dtype, *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype])
        self.x = [t(act, T, H, D) if H else None for H in (Hq, Hk)]
        self.dy = [t(act, T, H, D) if H else None for H in (Hq, Hk)]
        self.w = [t(par, D) if weights and norm else None for _ in range(2)]
        self.sections = sections or (rot // 2,)
        self.freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1)) if rot else np.zeros(0)
        self.pos = rng.integers(0, far, (len(self.sections), T))
        self.phi = O.angles(self.pos, self.freq, self.sections)
        self.interleaved, self.has_norm, self.offset = interleaved, norm, float(np.float32(offset))
        self.eps = float(np.float32(eps))
        gpu = lambda v: None if v is None else v.to(DEV)
        self.gx, self.gdy, self.gpos = [gpu(v) for v in self.x], [gpu(v) for v in self.dy], torch.from_numpy(self.pos).to(DEV)
        if not rot:
            self.gpos = None
        self.norm = nq.HeadNorm(D, act_dtype=DT[act], w_q=gpu(self.w[0]), w_k=gpu(self.w[1]),
                                inv_freq=torch.from_numpy(self.freq).to(DEV) if rot else None, interleaved=interleaved,
                                sections=self.sections, norm=norm, weight_offset=offset, eps=eps)

    def weight(self, i):
        return None if self.w[i] is None else f64(self.w[i]) + self.offset

    def near(self, got, want, mag, K):
        tol = K * E * mag
        tol = tol + half_step(got.dtype) * (np.abs(want) + tol) + 1e-42
        off = np.abs(f64(got) - want)
        assert np.all(off <= tol), float(np.max(off / tol))

    def check_forward(self, out):
        for i, (x, y) in enumerate(zip(self.x, out)):
            if x is None:
                assert y is None
                continue
            assert y.shape == x.shape and y.dtype == x.dtype
            want, mag = O.forward(f64(x), self.weight(i), self.phi, self.interleaved, self.eps, self.has_norm)
            self.near(y, want, mag, F)

    def forward(self, **kw):
        return nq.head_norm(*self.gx, self.gpos, self.norm, **kw)

    def backward(self, **kw):
        return nq.head_norm_backward(*self.gdy, *self.gx, self.gpos, self.norm, **kw)

    def check_backward(self, got):
        expect = set()
        for i, n in enumerate("qk"):
            if self.x[i] is None:
                continue
            dx, dw, DX, DW = O.backward(f64(self.dy[i]), f64(self.x[i]), self.weight(i), self.phi, self.interleaved,
                                        self.eps, self.has_norm)
            expect.add("d" + n)
            self.near(got["d" + n], dx, DX, GRAD)
            if self.w[i] is not None:
                expect.add("dw_" + n)
                T, H, _ = self.x[i].shape
                self.near(got["dw_" + n], dw, DW, GRAD + T * H + 64)
        assert set(got) == expect


SHAPES = [(2, 2), (4, 4), (8, 8), (8, 0), (16, 8), (64, 64), (64, 32), (64, 20), (72, 40), (80, 32), (80, 80), (96, 96),
          (100, 50), (100, 100), (126, 126), (128, 128), (128, 64), (128, 2), (128, 0), (130, 66), (192, 192), (200, 48),
          (256, 256), (256, 64), (300, 300), (384, 0), (510, 34), (512, 512)]


@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("act,par", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f16")])
def test_sizes(D, rot, interleaved, act, par):
    c = Case(3, 5, 2, D, rot, interleaved, act=act, par=par)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("D,rot", [(4, 0), (12, 8), (20, 20), (36, 34), (60, 12), (68, 64), (100, 96), (132, 132), (148, 10),
                                   (180, 60), (252, 252), (256, 100), (260, 260)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("act,par", [("f32", "bf16"), ("bf16", "f32")])
def test_multiples_of_four(D, rot, interleaved, act, par):
    """Heads and rotations that four divides and eight does not, some parts of a wider output
    that starts at an odd element."""
    c = Case(70, 7, 3, D, rot, interleaved, act=act, par=par)
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    wide = torch.zeros(70, 10 * D + 3, device=DEV, dtype=DT[act])
    q, k = wide[:, 1:1 + 7 * D].unflatten(1, (7, D)), wide[:, 2 + 7 * D:2 + 10 * D].unflatten(1, (3, D))
    q.copy_(c.gx[0]), k.copy_(c.gx[1])
    for got, want in zip(nq.head_norm(q, k, c.gpos if rot else None, c.norm), c.forward()):
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [0, 1, 2, 5, 63, 300, 2100])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 1), (64, 8), (3, 0), (0, 5), (9, 3), (1, 40)])
@pytest.mark.parametrize("D", [64, 100])
def test_tokens_and_heads(T, Hq, Hk, D):
    c = Case(T, Hq, Hk, D, act="bf16")
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("sections", [(32, 32), (10, 30, 24), (0, 64), (64, 0), (1, 2, 3, 58), (16, 16, 16, 16), (63, 0, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(sections, interleaved):
    c = Case(37, 3, 3, 128, sections=sections, interleaved=interleaved)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("norm,weights,offset,rot", [(False, False, 0.0, 128), (True, False, 0.0, 128), (True, True, 1.0, 64),
                                                     (True, False, 1.0, 0), (False, False, 0.0, 50)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_forms(norm, weights, offset, rot, act):
    c = Case(20, 4, 2, 128, rot, norm=norm, weights=weights, offset=offset, act=act)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


def test_far_positions():
    """2^24 radians and more.  The angle's error, 2^-52 phi for the product and as much
    for the turns, stays below e up to 2^27; at 2^31 it is 2^-20."""
    for far, K in ((2 ** 24, F), (2 ** 31, F + 32)):
        c = Case(50, 2, 2, 128, far=far, seed=4)
        c.pos[:] = far - 1 - np.arange(50)
        c.gpos.copy_(torch.from_numpy(c.pos))
        c.phi = O.angles(c.pos, c.freq, c.sections)
        for i, y in enumerate(c.forward()):
            want, mag = O.forward(f64(c.x[i]), c.weight(i), c.phi, False, c.eps)
            c.near(y, want, mag, K)


def test_negative_positions_turn_back():
    c = Case(9, 2, 2, 64, norm=False)
    q, k = c.forward()
    c.gpos.neg_()
    c.gx = [q, k]
    for x, y in zip(c.x, c.forward()):
        c.near(y, f64(x), 2 * O.spread(f64(x), c.phi, False), 2 * F)


def test_parts_of_a_fused_output():
    """q, k and v side by side in one linear's output, rows at any element."""
    rng = np.random.default_rng(5)
    for D, Hq, Hk in ((128, 8, 2), (100, 3, 1)):
        for pad in (0, 1, 8):
            for act in ("bf16", "f32"):
                c = Case(33, Hq, Hk, D, act=act)
                wide = torch.from_numpy(rng.standard_normal((33, (Hq + Hk) * D + pad)).astype(np.float32)).to(DT[act]).to(DEV)
                q, k = wide[:, pad:pad + Hq * D].unflatten(1, (Hq, D)), wide[:, pad + Hq * D:].unflatten(1, (Hk, D))
                c.gx, c.x = [q, k], [q.cpu(), k.cpu()]
                c.check_forward(c.forward())
                c.check_backward(c.backward())


def test_in_place():
    c = Case(40, 8, 2, 128, act="bf16")
    want = c.forward()
    mine = [t.clone() for t in c.gx]
    got = nq.head_norm(*mine, c.gpos, c.norm, inplace=True)
    assert all(g is m and torch.equal(g, w) for g, m, w in zip(got, mine, want))
    want = c.backward()
    grads = [t.clone() for t in c.gdy]
    got = nq.head_norm_backward(*grads, *c.gx, c.gpos, c.norm, inplace=True)
    assert got["dq"] is grads[0] and got["dk"] is grads[1]
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_rows_that_are_not_finite_stay_alone():
    c = Case(6, 4, 2, 96, act="f32")
    for x in c.gx:
        x[1, 0, 3], x[2, 1, 5], x[3, 0] = float("inf"), float("nan"), 0.0
    out = c.forward()
    for i, y in enumerate(out):
        bad = torch.zeros(y.shape[:2], dtype=torch.bool)
        bad[1, 0] = bad[2, 1] = True
        finite = torch.isfinite(y).all(-1).cpu()
        assert torch.equal(finite, ~bad)
        assert not y[3, 0].any()
        want, mag = O.forward(f64(c.x[i]), c.weight(i), c.phi, False, c.eps)
        keep = ~bad.numpy()
        keep[3, 0] = False
        tol = F * E * mag + half_step(y.dtype) * np.abs(want) * (1 + 1e-6) + 1e-42
        assert np.all((np.abs(f64(y) - want) <= tol)[keep])


def test_gradients_are_the_slope():
    """The slope of sum(y g) along a direction of x and of the weights, by differences of
    the oracle (their error under 1e-6 of the norms' product)."""
    c = Case(7, 3, 2, 80, 32, sections=(6, 10))
    got = c.backward()
    rng = np.random.default_rng(2)
    for i, n in enumerate("qk"):
        x, w, g = f64(c.x[i]), c.weight(i), f64(c.dy[i])
        loss = lambda x, w: float(np.sum(g * O.forward(x, w, c.phi, False, c.eps)[0]))
        way, step = rng.standard_normal(x.shape), 1e-5
        slope = (loss(x + step * way, w) - loss(x - step * way, w)) / (2 * step)
        assert abs(slope - np.sum(f64(got["d" + n]) * way)) <= 1e-5 * np.linalg.norm(f64(got["d" + n])) * np.linalg.norm(way)
        way = rng.standard_normal(w.shape)
        slope = (loss(x, w + step * way) - loss(x, w - step * way)) / (2 * step)
        assert abs(slope - np.sum(f64(got["dw_" + n]) * way)) <= 1e-5 * np.linalg.norm(f64(got["dw_" + n])) * np.linalg.norm(way)


def test_repeated_calls_give_the_same_bits():
    c = Case(900, 16, 4, 128, act="bf16")
    a, b = c.backward(), c.backward()
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("T", [1, 70])
def test_captured_and_replayed(T):
    c = Case(T, 8, 2, 128, act="bf16")
    side = torch.cuda.Stream()

    def both():
        q, k = c.forward()
        return {"q": q, "k": k, **c.backward()}
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kept = both()
    gen = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(3):
        for t in (*c.gx, *c.gdy):
            t.copy_(torch.randn(t.shape, device=DEV, generator=gen))
        c.gpos.copy_(torch.randint(0, 9999, c.gpos.shape, device=DEV, generator=gen))
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(kept[n], want[n]) for n in want)


# ------------------------------------------------------------------ into the cache
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 20, True), (96, 96, True), (128, 128, False),
                                               (128, 50, False), (192, 64, False), (256, 256, True), (256, 66, False)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_write_is_norm_then_write(kind, D, rot, interleaved, act):
    """The cache's bytes and q' are those of head_norm and kv_write one after the other."""
    for T, Hq, Hk in ((1, 8, 2), (5, 3, 3), (70, 8, 1), (3, 20, 5)):
        c = Case(T, Hq, Hk, D, rot, interleaved, act=act)
        v = torch.randn(T, Hk, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).to(DT[act])
        a, b = (nq.KvCache(6, Hk, D, page=16, kind=kind, device=DEV) for _ in range(2))
        a.data.fill_(7), b.data.fill_(7)
        slots = torch.randperm(96, device=DEV)[:T]
        slots[T // 2] = -1
        q, k = c.forward()
        nq.kv_write(k, v, a, slots)
        got = nq.head_norm_write(*c.gx, v, c.gpos, c.norm, b, slots)
        assert torch.equal(got, q) and torch.equal(a.data, b.data)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("D,rot", [(64, 4), (96, 92), (128, 100), (192, 180), (256, 252)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write_of_rotations_that_four_divides(kind, D, rot, interleaved):
    for act in ("bf16", "f32"):
        c = Case(70, 9, 5, D, rot, interleaved, act=act)
        v = torch.randn(70, 5, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(D)).to(DT[act])
        a, b = (nq.KvCache(6, 5, D, page=16, kind=kind, device=DEV) for _ in range(2))
        a.data.fill_(7), b.data.fill_(7)
        slots = torch.randperm(96, device=DEV)[:70]
        q, k = c.forward()
        nq.kv_write(k, v, a, slots)
        got = nq.head_norm_write(*c.gx, v, c.gpos, c.norm, b, slots)
        assert torch.equal(got, q) and torch.equal(a.data, b.data)
