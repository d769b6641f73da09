"""The binding's checks of 4-bit linears and block norms, without a GPU: stand-ins
with a tensor's attributes reach every check, and none of them is dereferenced."""
import pytest
import torch

import binary_rank_gemv_packed_amd as nq

GPU = torch.device("cuda", 0)


class Stand:
    """What the binding asks of a tensor that lies on a GPU."""

    def __init__(self, shape, dtype, device=GPU, contiguous=True):
        self.shape, self.dtype, self.device, self._contiguous = torch.Size(shape), dtype, device, contiguous
        self.is_cuda = device.type == "cuda"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 0x7F0000000000


ROWS, D = 4, 64
BAD_SCRATCH = [Stand((1 << 20,), torch.uint8, torch.device("cpu")), Stand((1 << 20,), torch.uint8, torch.device("cuda", 1)),
               Stand((1 << 20,), torch.float32), Stand((1 << 20,), torch.uint8, contiguous=False)]


@pytest.mark.parametrize("ws", BAD_SCRATCH, ids=["host", "other device", "dtype", "strided"])
def test_norm_backward_refuses_a_workspace_of_another_kind(ws):
    """A host pointer or a strided view (whose numel counts bytes that it does not own)
    must not reach the kernels."""
    f32 = torch.float32
    norm = nq.BlockNorm(D, act_dtype=f32)
    t = [Stand((ROWS, D), f32) for _ in range(4)]
    with pytest.raises(nq.NQError, match="workspace"):
        nq.block_norm_backward(t[0], t[1], t[2], t[3], Stand((2, ROWS), f32), norm, workspace=ws)


def test_unpack_refuses_outputs_on_each_other():
    """Codes (64 x 96 bytes) and zero points (64 x 3 bytes) written into one another."""
    import ctypes
    fake, far = 0x7F0000000000, 0x7F0040000000
    lay = nq.nq_q4_layer(64, 96, 32, nq.NQ_F16, 1, fake)
    for zeros in (far, far + 64 * 96 - 1, far - 64 * 3 + 1):
        assert nq.lib().nq_q4_unpack(ctypes.byref(lay), far, zeros, None) == nq.NQ_ERR_INVALID_ARG
        assert b"overlap" in nq.lib().nq_last_error()
