"""GPU: block norms and their gradients against the fp64 oracle.

Tolerances (derived, not fitted), with e = 2^-24 and K = 64.  A sum over a row is
at most 32 sums in a thread, 6 in a wave and 16 over waves, each off by e of a
partial sum of positive terms, so 1/rms is off by under (54 + 3) / 2 e of
itself and a value of u, of h' or of x by under K e of the magnitudes it is made
of; x also sees what h' is off by.  In the backward pass each mean is off by 57 e
of the mean of magnitudes; a gradient through both norms by 3 K e of the
magnitudes; a sum over R rows by another (R + 16) e.  An output is rounded once,
by half a step of its type (bf16: 2^-8, fp32: 2^-24 of the value)."""
import numpy as np
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from oracle import nq_norm as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
E, K = 2.0 ** -24, 64
A, B, EPS = 0.9, 0.7, 1e-5


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, rows, d, act="bf16", res="f32", par="f32", gate=None, post=True, pre=True, weights=True,
                 block=True, offset=0.0, seed=0):
        rng = np.random.default_rng([seed, rows, d, post, pre])
        t = lambda dtype, *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype])
        self.h, self.y = t(res, rows, d), t(act, rows, d) if block else None
        self.dx, self.dh = t(act, rows, d) if pre else None, t(res, rows, d)
        self.wp = t(par, d) if weights and post else None
        self.wq = t(par, d) if weights and pre else None
        self.gate = t(par, d) if gate == "channel" else t(act, rows, d) if gate == "rows" else None
        self.rows_gate = gate == "rows"
        self.post, self.pre, self.offset, self.d = post, pre, offset, d
        gpu = lambda v: None if v is None else v.to(DEV)
        self.norm = nq.BlockNorm(d, act_dtype=DT[act], res_dtype=DT[res], w_post=gpu(self.wp), w_pre=gpu(self.wq),
                                 gate=gpu(self.gate) if gate == "channel" else None, post=post, pre=pre, res_scale=A,
                                 block_scale=B, weight_offset=offset, eps=EPS)
        self.gpu = {k: gpu(getattr(self, k)) for k in ("h", "y", "dx", "dh")}
        self.gpu["gate"] = gpu(self.gate) if self.rows_gate else None
        # the scales as the kernels hold them
        self.a, self.b, self.eps, self.off = (float(np.float32(v)) for v in (A, B, EPS, offset))

    def weight(self, w):
        return None if w is None else f64(w) + self.off

    def forward(self, **kw):
        return nq.block_norm(self.gpu["h"], self.gpu["y"], self.norm, gate=self.gpu["gate"], **kw)

    def reference(self):
        return N.forward(f64(self.h), f64(self.y), self.weight(self.wp), self.weight(self.wq), f64(self.gate), self.a,
                         self.b, self.eps, self.post, self.pre)

    def check_forward(self, h_out, x):
        ref, xr = self.reference()
        err_h = np.zeros_like(ref)
        if self.y is not None:
            branch = np.abs(ref - self.a * f64(self.h))
            err_h = K * E * (np.abs(self.a * f64(self.h)) + branch)
            tol = err_h + half_step(h_out.dtype) * (np.abs(ref) + err_h) + 1e-42
            assert np.all(np.abs(f64(h_out) - ref) <= tol)
        if not self.pre:
            assert x is None
            return
        w = np.abs(self.weight(self.wq)) if self.wq is not None else 1.0
        relative = np.linalg.norm(err_h, axis=1, keepdims=True) / np.maximum(
            np.linalg.norm(ref, axis=1, keepdims=True), 1e-30)
        tol = N.rstd(ref, self.eps) * w * err_h + np.abs(xr) * (relative + K * E)
        tol = tol + half_step(x.dtype) * (np.abs(xr) + tol) + 1e-42
        assert np.all(np.abs(f64(x) - xr) <= tol)

    def backward(self, stats, h_out, **kw):
        return nq.block_norm_backward(self.gpu["dx"], kw.pop("dh", self.gpu["dh"]), h_out, self.gpu["y"], stats,
                                      self.norm, gate=self.gpu["gate"], **kw)

    def check_backward(self, got, stats, h_out, dh="given"):
        st = f64(stats)
        ref = N.backward(f64(self.dx), f64(self.dh) if dh == "given" else None, f64(h_out), f64(self.y),
                         self.weight(self.wp), self.weight(self.wq), f64(self.gate), self.a, self.b, st[0][:, None],
                         st[1][:, None], self.post, self.pre)
        M, R = ref["M"], self.h.shape[0]

        def near(name, want, mag, rows=0):
            t = got[name]
            tol = (3 * K + (rows + 16 if rows else 0)) * E * mag
            tol = tol + half_step(t.dtype) * (np.abs(want) + tol) + 1e-42
            assert np.all(np.abs(f64(t) - want) <= tol), (name, float(np.max(np.abs(f64(t) - want) / tol)))

        expect = {"dh"}
        near("dh", ref["h"], M["h"])
        if self.wq is not None:
            expect.add("dw_pre")
            near("dw_pre", ref["w_pre"], M["w_pre"], R)
        if self.y is not None:
            expect.add("dy")
            near("dy", ref["y"], M["y"])
            if self.wp is not None:
                expect.add("dw_post")
                near("dw_post", ref["w_post"], M["w_post"], R)
            if self.gate is not None:
                expect.add("dgate")
                if self.rows_gate:
                    near("dgate", ref["gate"], M["gate"])
                else:
                    near("dgate", ref["gate"].sum(0), M["gate"].sum(0), R)
        assert set(got) == expect


WIDTHS = [1, 2, 7, 8, 63, 64, 100, 513, 1619, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 28672, 32767, 32768]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "f32", "f16"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16")]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("act,res,par", TYPES)
@pytest.mark.parametrize("gate", [None, "channel", "rows"])
def test_widths(d, act, res, par, gate):
    c = Case(3, d, act, res, par, gate)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)


@pytest.mark.parametrize("rows", [1, 2, 511, 512, 513, 1100, 2500])
@pytest.mark.parametrize("d", [96, 1619, 2056])
@pytest.mark.parametrize("gate", [None, "channel", "rows"])
def test_row_counts(rows, d, gate):
    c = Case(rows, d, "bf16", "f32", "f32", gate)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)


def test_many_rows_of_a_wide_stream():
    for d in (8192, 9000):
        c = Case(700, d, "bf16", "bf16", "bf16", "channel")
        h_out, x, stats = c.forward(with_stats=True)
        c.check_forward(h_out, x)
        c.check_backward(c.backward(stats, h_out), stats, h_out)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "rows"])
@pytest.mark.parametrize("rows,d", [(5, 72), (600, 1001)])
def test_every_form(post, pre, weights, gate, rows, d):
    c = Case(rows, d, "bf16", "f32", "bf16", gate, post, pre, weights)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)
    if pre:
        c.check_backward(c.backward(stats, h_out, dh=None), stats, h_out, dh=None)


@pytest.mark.parametrize("rows,d", [(1, 8), (600, 1001), (3, 8192)])
def test_before_the_first_block(rows, d):
    c = Case(rows, d, block=False)
    h_out, x, stats = c.forward(with_stats=True)
    assert h_out is c.gpu["h"]
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)


def test_weight_offset():
    c = Case(40, 500, "bf16", "bf16", "bf16", "channel", offset=1.0)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)


def test_stats_are_the_reciprocal_roots():
    c = Case(30, 1000, "f32", "f32")
    h_out, _, stats = c.forward(with_stats=True)
    ref, _ = c.reference()
    for got, v in ((stats[0], f64(c.y)), (stats[1], ref)):
        want = N.rstd(v, c.eps)[:, 0]
        assert np.all(np.abs(f64(got) - want) <= K * E * want)


@pytest.mark.parametrize("d", [96, 1001])
def test_in_place(d):
    c = Case(20, d, "bf16", "bf16", "bf16", "channel")
    h_out, x, stats = c.forward(with_stats=True)
    stream = c.gpu["h"].clone()
    out, x2 = nq.block_norm(stream, c.gpu["y"], c.norm, inplace=True)
    assert out is stream and torch.equal(stream, h_out) and torch.equal(x, x2)
    apart = c.backward(stats, h_out)
    dh = c.gpu["dh"].clone()
    over = c.backward(stats, h_out, dh=dh, inplace=True)
    assert over["dh"] is dh
    for k in apart:
        assert torch.equal(apart[k], over[k]), k


def test_zero_rows_of_values_and_no_rows():
    c = Case(4, 200, "f32", "f32", gate="channel")
    c.y[1], c.h[2] = 0, 0
    c.y[3], c.h[3] = 0, 0
    c.gpu["y"], c.gpu["h"] = c.y.to(DEV), c.h.to(DEV)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    assert not x[3].any()
    c.check_backward(c.backward(stats, h_out), stats, h_out)
    c = Case(0, 200, "f32", "f32", gate="channel")
    h_out, x, stats = c.forward(with_stats=True)
    assert h_out.shape == x.shape == (0, 200)
    got = c.backward(stats, h_out)
    for k in ("dw_pre", "dw_post", "dgate"):
        assert got[k].shape == (200,) and not got[k].any()


def test_nan_and_infinity_stay_in_their_row():
    c = Case(6, 300, "bf16", "f32", gate="rows")
    clean = c.forward()
    c.gpu["y"][1, 7], c.gpu["y"][4, 0] = float("nan"), float("inf")
    dirty = c.forward()
    keep = [0, 2, 3, 5]
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
        assert torch.isnan(b[1]).all()


def test_repeated_calls_give_identical_bits():
    c = Case(1500, 1001, "bf16", "f32", gate="channel")
    h_out, x, stats = c.forward(with_stats=True)
    first = c.backward(stats, h_out)
    for _ in range(4):
        again = c.backward(stats, h_out)
        for k in first:
            assert torch.equal(first[k], again[k]), k


@pytest.mark.parametrize("off", [1, 4, 8])
def test_unaligned_tensors_and_what_lies_round_them(off):
    """Views that start `off` values into their storage; the storage round the
    outputs and the rest of the workspace keep their contents."""
    for rows, d in ((5, 64), (600, 200), (3, 2001)):
        c = Case(rows, d, "bf16", "f32", "bf16", "rows")

        def moved(t):
            b = torch.full((t.numel() + 2 * off,), 3.0, dtype=t.dtype, device=DEV)
            v = b[off:off + t.numel()].view(t.shape)
            v.copy_(t)
            return b, v
        want = c.forward(with_stats=True)
        grads = c.backward(want[2], want[0])
        bases = {}
        for k in list(c.gpu):
            bases[k], c.gpu[k] = moved(c.gpu[k])
        base_h, h = moved(c.h.to(DEV))
        out, x, stats = nq.block_norm(h, c.gpu["y"], c.norm, gate=c.gpu["gate"], inplace=True, with_stats=True)
        for a, b in zip(want, (out, x, stats)):
            # the scalar path adds in another order
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-5)
        assert bool((base_h[:off] == 3).all()) and bool((base_h[-off:] == 3).all())
        need = nq.lib().nq_block_norm_workspace_bytes(c.norm.ref, rows)
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        got = c.backward(stats, out, inplace=True, workspace=ws)
        c.check_backward(got, stats, out)
        assert bool((ws[need:] == 0xA5).all())
        assert bool((bases["dh"][:off] == 3).all()) and bool((bases["dh"][-off:] == 3).all())
        assert set(got) == set(grads)


def test_on_another_stream():
    c = Case(600, 2048, "bf16", "f32", gate="channel")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    h_out, x, stats = c.forward(with_stats=True, stream=stream)
    got = c.backward(stats, h_out, stream=stream)
    junk = [torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(8)]
    stream.synchronize()
    c.check_forward(h_out, x)
    c.check_backward(got, stats, h_out)
    del junk


@pytest.mark.parametrize("gate", [None, "channel", "rows"])
def test_gradients_against_differences(gate):
    """The kernels' forward, moved along a direction, against the kernels'
    gradient.  L = sum(x dx) + sum(h' dh) in fp64 of fp32 outputs; with a step of
    2^-7 the third derivative leaves about step^2 of L's scale and the outputs'
    rounding about K 2^-24 / step of it: under 1e-3 of the sum of magnitudes."""
    c = Case(8, 96, "f32", "f32", "f32", gate)
    h_out, x, stats = c.forward(with_stats=True)
    got = c.backward(stats, h_out)
    rng = np.random.default_rng(9)

    def loss(h, y, wp, wq, g):
        channel = gate == "channel"
        norm = nq.BlockNorm(96, act_dtype=torch.float32, w_post=wp, w_pre=wq, gate=g if channel else None, res_scale=A,
                            block_scale=B, eps=EPS)
        ho, xx = nq.block_norm(h, y, norm, gate=None if channel else g)
        return float((ho.double() * c.gpu["dh"].double()).sum() + (xx.double() * c.gpu["dx"].double()).sum())

    params = {"dh": c.gpu["h"], "dy": c.gpu["y"], "dw_post": c.wp.to(DEV), "dw_pre": c.wq.to(DEV),
              "dgate": c.gate.to(DEV) if gate else None}
    for k, p in params.items():
        if p is None:
            continue
        step = 2.0 ** -7
        way = torch.from_numpy(rng.choice([-1.0, 1.0], p.shape)).float().to(DEV)
        ends = [loss(*[v + sign * step * way if n == k else v for n, v in params.items()]) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        want = float((got[k].double() * way.double()).sum())
        scale = float(got[k].double().abs().sum())
        assert abs(slope - want) <= 1e-3 * scale, (k, slope, want, scale)


def test_binding_refusals():
    c = Case(4, 64, "bf16", "f32", "f32", "channel")
    h, y, st = c.gpu["h"], c.gpu["y"], torch.empty(2, 4, device=DEV)
    for bad in (lambda: nq.block_norm(h.bfloat16(), y, c.norm), lambda: nq.block_norm(h, y.float(), c.norm),
                lambda: nq.block_norm(h, y[:3], c.norm), lambda: nq.block_norm(h[:, :32], y, c.norm),
                lambda: nq.block_norm(h.cpu(), y, c.norm), lambda: nq.block_norm(h, y.cpu(), c.norm),
                lambda: nq.block_norm(h.t().contiguous().t(), y, c.norm),
                lambda: nq.block_norm(h, y, c.norm, gate=y),
                lambda: nq.block_norm_backward(y, h, h, y, st[:, :3], c.norm),
                lambda: nq.block_norm_backward(None, h, h, y, st, c.norm),
                lambda: nq.block_norm_backward(y, None, h, y, st, c.norm, inplace=True),
                lambda: nq.BlockNorm(64, w_post=torch.ones(32, device=DEV)),
                lambda: nq.BlockNorm(64, w_post=torch.ones(64, device=DEV), gate=torch.ones(64, device=DEV).half()),
                lambda: nq.BlockNorm(64, w_post=torch.ones(64, device=DEV).double())):
        with pytest.raises(nq.NQError):
            bad()
