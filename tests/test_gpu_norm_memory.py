"""GPU: block norms on either side of the backward pass's 256 workgroups, and with
every tensor, those that the binding would allocate among them, at any element and
with guarded storage around it (through the C ABI)."""
import pytest
import torch

import binary_rank_gemv_packed_amd as nq
from tests.test_gpu_norm import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [254, 255, 256, 257, 258, 767, 768, 769])
@pytest.mark.parametrize("d", [8, 96, 1619, 4104])
@pytest.mark.parametrize("gate", [None, "channel", "rows"])
def test_rows_around_the_workgroups(rows, d, gate):
    c = Case(rows, d, "bf16", "f32", "f32", gate)
    h_out, x, stats = c.forward(with_stats=True)
    c.check_forward(h_out, x)
    c.check_backward(c.backward(stats, h_out), stats, h_out)


class Guarded:
    """A (shape) view `off` values into storage that holds `fill` around it."""

    def __init__(self, shape, dtype, off, fill=3.0, values=None):
        n = torch.Size(shape).numel()
        self.base = torch.full((n + 2 * off,), fill, dtype=dtype, device=DEV)
        self.off, self.n, self.fill = off, n, fill
        self.v = self.base[off:off + n].view(shape)
        if values is not None:
            self.v.copy_(values)

    def untouched(self):
        around = torch.cat([self.base[:self.off], self.base[self.off + self.n:]])
        return bool((around == self.fill).all())


@pytest.mark.parametrize("off", [1, 3, 4, 8])
@pytest.mark.parametrize("rows,d", [(5, 64), (300, 200), (3, 2001), (2, 8192), (2, 8200), (2, 20001)])
@pytest.mark.parametrize("act,res", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("gate", ["channel", "rows"])
def test_every_tensor_at_any_element(off, rows, d, act, res, gate):
    c = Case(rows, d, act, res, "f32", gate)
    at, rt, f32 = c.gpu["y"].dtype, c.gpu["h"].dtype, torch.float32
    moved = {k: Guarded(v.shape, v.dtype, off, values=v) for k, v in c.gpu.items() if v is not None}
    c.gpu.update({k: g.v for k, g in moved.items()})
    out = {"h_out": Guarded((rows, d), rt, off), "x": Guarded((rows, d), at, off), "stats": Guarded((2, rows), f32, off)}
    p = lambda k: {**moved, **out}[k].v.data_ptr() if k in moved or k in out else None
    stream = torch.cuda.current_stream().cuda_stream
    assert nq.lib().nq_block_norm_fwd(c.norm.ref, rows, p("h"), p("y"), p("gate"), p("h_out"), p("x"), p("stats"),
                                      stream) == nq.NQ_OK
    c.check_forward(out["h_out"].v, out["x"].v)
    channel = gate == "channel"
    out |= {"dh_new": Guarded((rows, d), rt, off), "dy": Guarded((rows, d), at, off)}
    out |= {k: Guarded((d,), f32, off) for k in ("dw_post", "dw_pre")}
    out["dgate"] = Guarded((d,), f32, off) if channel else Guarded((rows, d), at, off)
    need = nq.lib().nq_block_norm_workspace_bytes(c.norm.ref, rows)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    assert nq.lib().nq_block_norm_bwd(
        c.norm.ref, rows, p("dx"), p("dh"), p("h_out"), p("y"), p("gate"), p("stats"), p("dh_new"), p("dy"),
        None if channel else p("dgate"), p("dw_post"), p("dw_pre"), p("dgate") if channel else None, ws.data_ptr(), need,
        stream) == nq.NQ_OK
    got = {"dh" if k == "dh_new" else k: out[k].v for k in ("dh_new", "dy", "dw_post", "dw_pre", "dgate")}
    c.check_backward(got, out["stats"].v, out["h_out"].v)
    assert bool((ws[need:] == 0xA5).all())
    for k, g in {**moved, **out}.items():
        assert g.untouched(), k
