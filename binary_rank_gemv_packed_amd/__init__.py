"""Python binding of libnq: linear layers with a low-rank binary-factorised weight
W_hat = diag(s1) U diag(g) V^T diag(s2) on MI355X, and what stands beside them in a
model: linears with 4-bit weights (q4_*) and the norms between blocks (block_norm).

Argument marshalling only: every step of the forward runs in the HIP kernels of
libnq.so, reached through its C ABI (include/nq.h).  PyTorch provides device
memory and the current stream.  There is no CPU fallback: if the library is not
built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnq.so")

NQ_OK, NQ_ERR_INVALID_ARG, NQ_ERR_NOT_PM1, NQ_ERR_WORKSPACE, NQ_ERR_UNSUPPORTED, NQ_ERR_HIP, NQ_ERR_INTERNAL, \
    NQ_ERR_RANGE = 0, -1, -2, -3, -4, -5, -6, -7
NQ_F32, NQ_F16, NQ_BF16 = 0, 1, 2
NQ_GROUP_MAX = 4  # layers per group call (include/nq.h)
NQ_ENVELOPE_MAX = 4  # terms of a rank-l envelope (include/nq.h)
NQ_NORM_POST, NQ_NORM_PRE, NQ_NORM_MAX_DIM = 1, 2, 32768  # block norms (include/nq.h)
PATHS = {"auto": 0, "gemv": 1, "gemm": 2, "valu": 3, "decode": 4}

_DT = {torch.float32: NQ_F32, torch.float16: NQ_F16, torch.bfloat16: NQ_BF16}
_ACT = (torch.bfloat16, torch.float32)  # of activations


class NQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libnq status {status}: {message}")
        self.status = status


class nq_layer(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("r", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("blob", ctypes.c_void_p)]


class nq_q4_layer(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("zeros", ctypes.c_int32), ("blob", ctypes.c_void_p)]


class nq_block_norm(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("flags", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("block_scale", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("gate", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libnq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with `python -m binary_rank_gemv_packed_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    c_int, c_size, vp = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    P, Q, N = ctypes.POINTER(nq_layer), ctypes.POINTER(nq_q4_layer), ctypes.POINTER(nq_block_norm)
    sigs = {
        "nq_abi_version": (c_int, []),
        "nq_layer_bytes": (c_size, [c_int, c_int, c_int, c_int]),
        "nq_pack_factors": (c_int, [P, vp, vp, vp, vp, vp, vp]),
        "nq_unpack_factors": (c_int, [P, vp, vp, vp]),
        "nq_transpose_layer": (c_int, [P, P, vp]),
        "nq_workspace_bytes": (c_size, [P, c_int]),
        "nq_workspace_bytes_path": (c_size, [P, c_int, c_int]),
        "nq_linear_fwd": (c_int, [P, vp, c_int, vp, c_int, c_int, vp, c_size, vp]),
        "nq_linear_fwd_path": (c_int, [P, vp, c_int, vp, c_int, c_int, vp, c_size, vp, c_int]),
        "nq_linear_fwd_profiled": (c_int, [P, vp, c_int, vp, c_int, c_int, vp, c_size, vp, c_int, vp, c_int,
                                           ctypes.POINTER(c_int), vp]),
        "nq_linear_fwd_noalloc": (c_int, [P, vp, c_int, vp, c_int, c_int, vp]),
        "nq_workspace_bytes_group": (c_size, [vp, c_int, c_int]),
        "nq_workspace_bytes_envelope": (c_size, [P, c_int, c_int]),
        "nq_linear_fwd_envelope": (c_int, [P, c_int, vp, vp, vp, c_int, vp, c_int, c_int, vp, c_size, vp]),
        "nq_linear_fwd_group": (c_int, [vp, c_int, vp, c_int, vp, c_int, c_int, vp, c_size, vp]),
        "nq_linear_fwd_group_profiled": (c_int, [vp, c_int, vp, c_int, vp, c_int, c_int, vp, c_size, vp, vp, c_int,
                                                 ctypes.POINTER(c_int), vp]),
        "nq_read_probe": (c_int, [vp, c_size, vp, vp, ctypes.POINTER(c_int)]),
        "nq_admm_workspace_bytes": (c_size, [c_int, c_int, c_int]),
        "nq_admm_factorize": (c_int, [vp, c_int, c_int, c_int, vp, vp, ctypes.c_float, c_int, c_int, vp, vp, vp, vp,
                                      vp, vp, vp, c_size, vp]),
        "nq_balance_scales": (c_int, [vp, vp, vp, c_int, c_int, c_int, vp]),
        "nq_q4_layer_bytes": (c_size, [c_int, c_int, c_int, c_int, c_int]),
        "nq_q4_pack": (c_int, [Q, vp, vp, vp, vp]),
        "nq_q4_unpack": (c_int, [Q, vp, vp, vp]),
        "nq_q4_workspace_bytes": (c_size, [Q, c_int]),
        "nq_q4_linear_fwd": (c_int, [Q, vp, c_int, vp, c_int, c_int, vp, c_size, vp]),
        "nq_q4_workspace_bytes_group": (c_size, [vp, c_int, c_int]),
        "nq_q4_linear_fwd_group": (c_int, [vp, c_int, vp, c_int, vp, c_int, c_int, vp, c_size, vp]),
        "nq_block_norm_fwd": (c_int, [N, c_int, vp, vp, vp, vp, vp, vp, vp]),
        "nq_block_norm_workspace_bytes": (c_size, [N, c_int]),
        "nq_block_norm_bwd": (c_int, [N, c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, c_size, vp]),
        "nq_bits_per_weight": (ctypes.c_double, [c_int, c_int, c_int, c_int]),
        "nq_rank_for_bits": (c_int, [c_int, c_int, ctypes.c_double, c_int]),
        "nq_status_string": (ctypes.c_char_p, [c_int]),
        "nq_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status: int) -> None:
    if status != NQ_OK:
        raise NQError(status, lib().nq_last_error().decode() or lib().nq_status_string(status).decode())


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _here(device: torch.device, stream):
    """The raw current stream, where a call needs no more than that: no stream
    given and `device` current (else None; 0 is the default stream).  torch's own
    raw form costs 0.1 us, building a Stream object to ask it 2.7 us, a third of a
    small launch."""
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        return torch._C._cuda_getCurrentRawStream(index)
    return None


def _on_stream(device: torch.device, stream, call):
    """call(raw stream) with `device` current: on the given stream, else on the
    device's current one.  What call allocates belongs to that stream."""
    raw = _here(device, stream)
    if raw is not None:
        return call(raw)
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream()
        if s.device != device:
            raise NQError(NQ_ERR_INVALID_ARG, f"stream on {s.device}, tensors on {device}")
        with torch.cuda.stream(s):
            return call(s.cuda_stream)


def _gpu_tensor(t: torch.Tensor, name: str, dtype, shape, device) -> None:
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise NQError(NQ_ERR_INVALID_ARG, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                                          f"{device} (got {t.dtype} {tuple(t.shape)} on {t.device})")


def _scratch(workspace: torch.Tensor, device) -> None:
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise NQError(NQ_ERR_INVALID_ARG, f"the workspace must be a contiguous uint8 tensor on {device}")


class Layer:
    """A packed layer: the device blob plus its dimensions."""

    def __init__(self, m: int, n: int, r: int, scale_dtype: torch.dtype, blob: torch.Tensor):
        self.m, self.n, self.r = m, n, r
        self.scale_dtype = scale_dtype
        self.blob = blob
        self.c = nq_layer(m, n, r, _DT[scale_dtype], blob.data_ptr())

    @property
    def ref(self):
        return ctypes.byref(self.c)

    @property
    def device(self):
        return self.blob.device


def layer_bytes(m: int, n: int, r: int, scale_dtype: torch.dtype = torch.float16) -> int:
    return int(lib().nq_layer_bytes(m, n, r, _DT[scale_dtype]))


def empty_layer(m: int, n: int, r: int, scale_dtype: torch.dtype = torch.float16, device="cuda") -> Layer:
    nbytes = layer_bytes(m, n, r, scale_dtype)
    if nbytes == 0:
        raise NQError(NQ_ERR_INVALID_ARG, f"invalid layer dimensions m={m} n={n} r={r}")
    return Layer(m, n, r, scale_dtype, torch.empty(nbytes, dtype=torch.uint8, device=device))


def pack(U: torch.Tensor, V: torch.Tensor, s1: torch.Tensor, g: torch.Tensor, s2: torch.Tensor,
         stream=None) -> Layer:
    """Packs int8 sign matrices U (m x r), V (n x r) and scales (fp16 or fp32,
    all of one dtype) already on the GPU.  Blocks until validation is done."""
    m, r = U.shape
    n, r2 = V.shape
    if r2 != r or s1.shape != (m,) or g.shape != (r,) or s2.shape != (n,):
        raise NQError(NQ_ERR_INVALID_ARG, "shape mismatch between U, V and the scale vectors")
    if U.dtype != torch.int8 or V.dtype != torch.int8:
        raise NQError(NQ_ERR_INVALID_ARG, "U and V must be int8")
    if not (s1.dtype == g.dtype == s2.dtype) or s1.dtype not in (torch.float16, torch.float32):
        raise NQError(NQ_ERR_INVALID_ARG, "scales must share one dtype, fp16 or fp32")
    U, V, s1, g, s2 = (t.contiguous() for t in (U, V, s1, g, s2))
    layer = empty_layer(m, n, r, s1.dtype, U.device)
    _check(lib().nq_pack_factors(layer.ref, U.data_ptr(), V.data_ptr(), s1.data_ptr(), g.data_ptr(),
                                 s2.data_ptr(), _stream(stream)))
    return layer


def unpack(layer: Layer, stream=None):
    """Sign matrices (U, V) read back from the packed blob, as int8 +-1."""
    U = torch.empty((layer.m, layer.r), dtype=torch.int8, device=layer.device)
    V = torch.empty((layer.n, layer.r), dtype=torch.int8, device=layer.device)
    _check(lib().nq_unpack_factors(layer.ref, U.data_ptr(), V.data_ptr(), _stream(stream)))
    return U, V


def transpose(layer: Layer, stream=None) -> Layer:
    """The layer of W_hat^T (U and V, s1 and s2 swapped, factors bit-transposed
    on the GPU): linear(dy, transpose(layer)) = dy W_hat, the backward product."""
    out = empty_layer(layer.n, layer.m, layer.r, layer.scale_dtype, device=layer.device)
    _check(lib().nq_transpose_layer(layer.ref, out.ref, _stream(stream)))
    return out


def workspace_bytes(layer: Layer, B: int, path: str = "auto") -> int:
    return int(lib().nq_workspace_bytes_path(layer.ref, B, PATHS[path]))


def new_workspace(layer: Layer, B: int) -> torch.Tensor:
    return torch.empty(max(workspace_bytes(layer, B), 256), dtype=torch.uint8, device=layer.device)


def linear_into(x: torch.Tensor, layer: Layer, y: torch.Tensor, workspace: torch.Tensor, path: str = "auto",
                stream=None) -> torch.Tensor:
    """y[B, m] = x[B, n] W_hat^T into caller buffers; enqueues on the stream and
    returns without synchronising (safe to capture in a graph)."""
    B = x.shape[0] if x.dim() == 2 else 1
    if x.dtype not in (torch.bfloat16, torch.float32) or y.dtype not in (torch.bfloat16, torch.float32):
        raise NQError(NQ_ERR_INVALID_ARG, "x and y must be bf16 or fp32")
    if not (x.is_contiguous() and y.is_contiguous()):
        raise NQError(NQ_ERR_INVALID_ARG, "x and y must be contiguous")
    if x.numel() != B * layer.n or y.numel() != B * layer.m:
        raise NQError(NQ_ERR_INVALID_ARG, "x or y has the wrong number of elements")
    _check(lib().nq_linear_fwd_path(layer.ref, x.data_ptr(), _DT[x.dtype], y.data_ptr(), _DT[y.dtype], B,
                                    workspace.data_ptr(), workspace.numel(), _stream(stream), PATHS[path]))
    return y


def linear_into_profiled(x: torch.Tensor, layer: Layer, y: torch.Tensor, workspace: torch.Tensor, events,
                         path: str = "auto", stream=None):
    """linear_into that records the given HIP events (raw hipEvent_t handles, as
    ints) around each kernel launch.  Returns [(workgroups, threads per
    workgroup)] of the launches, in order."""
    B = x.shape[0] if x.dim() == 2 else 1
    arr = (ctypes.c_void_p * len(events))(*events)
    dims = (ctypes.c_int32 * (2 * len(events)))()
    nl = ctypes.c_int32(0)
    _check(lib().nq_linear_fwd_profiled(layer.ref, x.data_ptr(), _DT[x.dtype], y.data_ptr(), _DT[y.dtype], B,
                                        workspace.data_ptr(), workspace.numel(), _stream(stream), PATHS[path],
                                        ctypes.cast(arr, ctypes.c_void_p), len(events), ctypes.byref(nl),
                                        ctypes.cast(dims, ctypes.c_void_p)))
    k = min(nl.value, len(events) - 1)
    return [(dims[2 * i], dims[2 * i + 1]) for i in range(k)]


def _group_arrays(layers, ys=None):
    refs = (ctypes.POINTER(nq_layer) * len(layers))(*[ctypes.pointer(L.c) for L in layers])
    yp = None if ys is None else (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    return refs, yp


def workspace_bytes_group(layers, B: int) -> int:
    refs, _ = _group_arrays(layers)
    return int(lib().nq_workspace_bytes_group(ctypes.cast(refs, ctypes.c_void_p), len(layers), B))


def _check_group(x, layers, ys):
    B = x.shape[0] if x.dim() == 2 else 1
    if len(ys) != len(layers):
        raise NQError(NQ_ERR_INVALID_ARG, "one output per layer")
    if x.dtype not in (torch.bfloat16, torch.float32) or any(y.dtype != ys[0].dtype for y in ys) or \
            ys[0].dtype not in (torch.bfloat16, torch.float32):
        raise NQError(NQ_ERR_INVALID_ARG, "x and the outputs must be bf16 or fp32 (one dtype for all outputs)")
    if not x.is_contiguous() or not all(y.is_contiguous() for y in ys):
        raise NQError(NQ_ERR_INVALID_ARG, "x and the outputs must be contiguous")
    if any(x.numel() != B * L.n for L in layers) or any(y.numel() != B * L.m for y, L in zip(ys, layers)):
        raise NQError(NQ_ERR_INVALID_ARG, "x or an output has the wrong number of elements")
    return B


def linear_group_into(x: torch.Tensor, layers, ys, workspace: torch.Tensor, stream=None):
    """ys[l] = x W_hat_l^T for layers sharing x (q/k/v, gate/up): two launches
    in all for B <= 4 (stage 1 over every layer's V^T, block-diagonal stage 2)."""
    B = _check_group(x, layers, ys)
    refs, yp = _group_arrays(layers, ys)
    _check(lib().nq_linear_fwd_group(ctypes.cast(refs, ctypes.c_void_p), len(layers), x.data_ptr(), _DT[x.dtype],
                                     ctypes.cast(yp, ctypes.c_void_p), _DT[ys[0].dtype], B, workspace.data_ptr(),
                                     workspace.numel(), _stream(stream)))
    return ys


def linear_group(x: torch.Tensor, layers, out_dtype: torch.dtype | None = None, stream=None):
    xx = x if x.dim() == 2 else x.view(1, -1)
    ys = [torch.empty((xx.shape[0], L.m), dtype=out_dtype or x.dtype, device=x.device) for L in layers]
    ws = torch.empty(max(workspace_bytes_group(layers, xx.shape[0]), 256), dtype=torch.uint8, device=x.device)
    linear_group_into(xx, layers, ys, ws, stream)
    return ys if x.dim() == 2 else [y.view(-1) for y in ys]


def linear_group_into_profiled(x: torch.Tensor, layers, ys, workspace: torch.Tensor, events, stream=None):
    """linear_group_into that records HIP events around each launch; returns
    [(workgroups, threads per workgroup)] of the launches."""
    B = _check_group(x, layers, ys)
    refs, yp = _group_arrays(layers, ys)
    arr = (ctypes.c_void_p * len(events))(*events)
    dims = (ctypes.c_int32 * (2 * len(events)))()
    nl = ctypes.c_int32(0)
    _check(lib().nq_linear_fwd_group_profiled(ctypes.cast(refs, ctypes.c_void_p), len(layers), x.data_ptr(),
                                              _DT[x.dtype], ctypes.cast(yp, ctypes.c_void_p), _DT[ys[0].dtype], B,
                                              workspace.data_ptr(), workspace.numel(), _stream(stream),
                                              ctypes.cast(arr, ctypes.c_void_p), len(events), ctypes.byref(nl),
                                              ctypes.cast(dims, ctypes.c_void_p)))
    k = min(nl.value, len(events) - 1)
    return [(dims[2 * i], dims[2 * i + 1]) for i in range(k)]


def linear_envelope(x: torch.Tensor, layer: Layer, s1_env: torch.Tensor, s2_env: torch.Tensor,
                    out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y = x W_hat^T with W_hat = sum_t diag(s1_env[t]) U diag(g) V^T diag(s2_env[t])
    (rank-l envelope; U, V, g from the layer): B x terms <= 4."""
    xx = x if x.dim() == 2 else x.view(1, -1)
    B, env = xx.shape[0], s1_env.shape[0]
    if s1_env.shape != (env, layer.m) or s2_env.shape != (env, layer.n) or \
            s1_env.dtype != layer.scale_dtype or s2_env.dtype != layer.scale_dtype:
        raise NQError(NQ_ERR_INVALID_ARG, "envelope scales must be (terms, m) and (terms, n) in the layer's dtype")
    if not (xx.is_contiguous() and s1_env.is_contiguous() and s2_env.is_contiguous()):
        raise NQError(NQ_ERR_INVALID_ARG, "x and the envelope scales must be contiguous")
    y = torch.empty((B, layer.m), dtype=out_dtype or x.dtype, device=x.device)
    ws = torch.empty(max(int(lib().nq_workspace_bytes_envelope(layer.ref, env, B)), 256), dtype=torch.uint8,
                     device=x.device)
    _check(lib().nq_linear_fwd_envelope(layer.ref, env, s1_env.data_ptr(), s2_env.data_ptr(), xx.data_ptr(),
                                        _DT[xx.dtype], y.data_ptr(), _DT[y.dtype], B, ws.data_ptr(), ws.numel(),
                                        _stream(stream)))
    return y if x.dim() == 2 else y.view(-1)


def linear_noalloc_into(x: torch.Tensor, layer: Layer, y: torch.Tensor, stream=None) -> torch.Tensor:
    """linear_into without a workspace: the library's static device scratch is
    used (see nq_linear_fwd_noalloc; calls overlapping on one GPU race)."""
    B = x.shape[0] if x.dim() == 2 else 1
    if x.dtype not in (torch.bfloat16, torch.float32) or y.dtype not in (torch.bfloat16, torch.float32):
        raise NQError(NQ_ERR_INVALID_ARG, "x and y must be bf16 or fp32")
    if not (x.is_contiguous() and y.is_contiguous()):
        raise NQError(NQ_ERR_INVALID_ARG, "x and y must be contiguous")
    if x.numel() != B * layer.n or y.numel() != B * layer.m:
        raise NQError(NQ_ERR_INVALID_ARG, "x or y has the wrong number of elements")
    _check(lib().nq_linear_fwd_noalloc(layer.ref, x.data_ptr(), _DT[x.dtype], y.data_ptr(), _DT[y.dtype], B,
                                       _stream(stream)))
    return y


def linear(x: torch.Tensor, layer: Layer, out_dtype: torch.dtype | None = None, path: str = "auto",
           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x W_hat^T for x of shape (B, n) or (n,); y has x's dtype unless given."""
    squeeze = x.dim() == 1
    x2 = x.reshape(1, -1) if squeeze else x
    x2 = x2.contiguous()
    B = x2.shape[0]
    y = torch.empty((B, layer.m), dtype=out_dtype or x.dtype, device=x.device)
    if workspace is None:
        workspace = new_workspace(layer, B)
    linear_into(x2, layer, y, workspace, path, stream)
    return y[0] if squeeze else y


def read_probe(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> tuple[int, int]:
    """Reads buf once (a measurement aid; see nq_read_probe) and XORs its
    32-bit words into sink[0] (int32, on buf's device).  Returns the launch's
    (workgroups, threads per workgroup)."""
    if not buf.is_contiguous() or sink.dtype != torch.int32 or sink.numel() < 1:
        raise NQError(NQ_ERR_INVALID_ARG, "buf must be contiguous and sink an int32 tensor")
    grid = (ctypes.c_int32 * 2)()
    _check(lib().nq_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(), _stream(stream),
                               grid))
    return int(grid[0]), int(grid[1])


def admm_factorize(W: torch.Tensor, A0: torch.Tensor, B0: torch.Tensor, rho: float, iters: int,
                   power_iters: int, with_err: bool = True, stream=None):
    """Initialiser of the binary factors of a dense fp32 weight W (m x n) from
    latent factors A0 (m x r), B0 (n x r), all on the GPU (nq_admm_factorize).
    Returns (U int8 m x r, V int8 n x r, s1, g, s2 fp32, err fp32 [iters + 1]
    or None)."""
    m, n = W.shape
    r = A0.shape[1]
    if A0.shape != (m, r) or B0.shape != (n, r):
        raise NQError(NQ_ERR_INVALID_ARG, f"A0 {tuple(A0.shape)} / B0 {tuple(B0.shape)} do not match W {m}x{n}, r={r}")
    for t in (W, A0, B0):
        if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
            raise NQError(NQ_ERR_INVALID_ARG, "W, A0 and B0 must be contiguous fp32 GPU tensors")
    dev = W.device
    need = int(lib().nq_admm_workspace_bytes(m, n, r))
    if need == 0:
        raise NQError(NQ_ERR_INVALID_ARG, f"invalid dimensions m={m} n={n} r={r}")
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    U = torch.empty(m, r, dtype=torch.int8, device=dev)
    V = torch.empty(n, r, dtype=torch.int8, device=dev)
    s1 = torch.empty(m, dtype=torch.float32, device=dev)
    g = torch.empty(r, dtype=torch.float32, device=dev)
    s2 = torch.empty(n, dtype=torch.float32, device=dev)
    err = torch.empty(iters + 1, dtype=torch.float32, device=dev) if with_err else None
    _check(lib().nq_admm_factorize(W.data_ptr(), m, n, r, A0.data_ptr(), B0.data_ptr(), float(rho), iters,
                                   power_iters, U.data_ptr(), V.data_ptr(), s1.data_ptr(), g.data_ptr(),
                                   s2.data_ptr(), err.data_ptr() if err is not None else None, ws.data_ptr(),
                                   ws.numel(), _stream(stream)))
    return U, V, s1, g, s2, err


def balance_scales(s1: torch.Tensor, g: torch.Tensor, s2: torch.Tensor, stream=None) -> None:
    """Power-of-two magnitude balancing of fp32 GPU scale vectors, in place
    (nq_balance_scales)."""
    for t in (s1, g, s2):
        if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
            raise NQError(NQ_ERR_INVALID_ARG, "s1, g and s2 must be contiguous fp32 GPU tensors")
    _check(lib().nq_balance_scales(s1.data_ptr(), g.data_ptr(), s2.data_ptr(), s1.numel(), s2.numel(), g.numel(),
                                   _stream(stream)))


# ------------------------------------------------------------------ 4-bit linears
class Q4Layer:
    """A packed 4-bit layer: the device blob plus its dimensions."""

    def __init__(self, m: int, n: int, group: int, scale_dtype: torch.dtype, zeros: bool, blob: torch.Tensor):
        self.m, self.n, self.group, self.scale_dtype, self.zeros, self.blob = m, n, group, scale_dtype, zeros, blob
        self.device = blob.device
        self.c = nq_q4_layer(m, n, group, _DT[scale_dtype], int(zeros), blob.data_ptr())
        self.ref = ctypes.byref(self.c)


class Q4Group:
    """4-bit layers that read the same x (q, k and v; gate and up): same n, group,
    scale dtype and kind of zero point, on one device."""

    def __init__(self, layers):
        self.layers = list(layers)
        if not 1 <= len(self.layers) <= NQ_GROUP_MAX or len({L.device for L in self.layers}) != 1:
            raise NQError(NQ_ERR_INVALID_ARG, f"a group holds 1..{NQ_GROUP_MAX} layers on one device")
        self.n, self.device = self.layers[0].n, self.layers[0].device
        self._refs = (ctypes.POINTER(nq_q4_layer) * len(self.layers))(*[ctypes.pointer(L.c) for L in self.layers])
        self.ref = ctypes.cast(self._refs, ctypes.c_void_p)

    def __len__(self):
        return len(self.layers)


def q4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, group: int = 128,
            stream=None) -> Q4Layer:
    """Packs the 4-bit weight W[i, j] = scales[i, j // group] * (codes[i, j] -
    zeros[i, j // group]) already on the GPU: codes uint8 (m, n) in 0..15, scales
    fp16 or fp32 (m, ceil(n / group)) and below 2^80 where finite, zeros uint8 of that
    shape in 0..15 or None for 8 everywhere; group 32, 64 or 128.  Blocks until
    validation is done."""
    if codes.dim() != 2 or codes.dtype != torch.uint8 or not codes.is_cuda:
        raise NQError(NQ_ERR_INVALID_ARG, "codes must be a uint8 GPU matrix")
    if scales.dtype not in (torch.float16, torch.float32):
        raise NQError(NQ_ERR_INVALID_ARG, "scales must be fp16 or fp32")
    m, n = codes.shape
    nbytes = int(lib().nq_q4_layer_bytes(m, n, group, _DT[scales.dtype], int(zeros is not None)))
    if nbytes == 0:
        raise NQError(NQ_ERR_INVALID_ARG, f"invalid 4-bit layer m={m} n={n} group={group}")

    def call(s):
        c, sc = codes.contiguous(), scales.contiguous()
        z = zeros.contiguous() if zeros is not None else None
        shape = torch.Size((m, (n + group - 1) // group))
        _gpu_tensor(sc, "scales", scales.dtype, shape, codes.device)
        if z is not None:
            _gpu_tensor(z, "zeros", torch.uint8, shape, codes.device)
        layer = Q4Layer(m, n, group, scales.dtype, z is not None,
                        torch.empty(nbytes, dtype=torch.uint8, device=codes.device))
        _check(lib().nq_q4_pack(layer.ref, c.data_ptr(), sc.data_ptr(), z.data_ptr() if z is not None else None, s))
        return layer

    return _on_stream(codes.device, stream, call)


def q4_unpack(layer: Q4Layer, stream=None):
    """(codes, zeros or None) read back from the packed blob, as q4_pack took them."""
    def call(s):
        codes = torch.empty((layer.m, layer.n), dtype=torch.uint8, device=layer.device)
        zeros = torch.empty((layer.m, (layer.n + layer.group - 1) // layer.group), dtype=torch.uint8,
                            device=layer.device) if layer.zeros else None
        _check(lib().nq_q4_unpack(layer.ref, codes.data_ptr(), zeros.data_ptr() if layer.zeros else None, s))
        return codes, zeros

    return _on_stream(layer.device, stream, call)


def q4_workspace_bytes(layer, B: int) -> int:
    """Workspace of q4_linear_into (a Q4Layer) or q4_linear_group_into (a Q4Group
    or a list of layers) for batch B."""
    if isinstance(layer, Q4Layer):
        return int(lib().nq_q4_workspace_bytes(layer.ref, B))
    group = layer if isinstance(layer, Q4Group) else Q4Group(layer)
    return int(lib().nq_q4_workspace_bytes_group(group.ref, len(group), B))


def new_q4_workspace(layer, B: int) -> torch.Tensor:
    device = layer.device if isinstance(layer, (Q4Layer, Q4Group)) else layer[0].device
    return torch.empty(max(q4_workspace_bytes(layer, B), 256), dtype=torch.uint8, device=device)


def _q4_batch(x: torch.Tensor, n: int, device) -> int:
    shape = x.shape
    if x.dtype not in _ACT or x.device != device or not x.is_contiguous() or len(shape) not in (1, 2) or \
            shape[-1] != n:
        raise NQError(NQ_ERR_INVALID_ARG, f"x must be contiguous bf16 or fp32 of shape (B, {n}) or ({n},) on {device}")
    return shape[0] if len(shape) == 2 else 1


def _q4_output(x: torch.Tensor, B: int, y: torch.Tensor, m: int, dtype: torch.dtype) -> None:
    if dtype not in _ACT:
        raise NQError(NQ_ERR_INVALID_ARG, "y must be bf16 or fp32")
    _gpu_tensor(y, "y", dtype, (B, m) if x.dim() == 2 else (m,), x.device)


def q4_linear_into(x: torch.Tensor, layer: Q4Layer, y: torch.Tensor, workspace: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """y = x W^T into caller buffers, x (B, n) or (n,) bf16 or fp32, y (B, m) or
    (m,); enqueues on the stream and returns without synchronising (safe to
    capture in a graph)."""
    device = layer.device
    B = _q4_batch(x, layer.n, device)
    _q4_output(x, B, y, layer.m, y.dtype)
    _scratch(workspace, device)
    _on_stream(device, stream, lambda s: _check(lib().nq_q4_linear_fwd(
        layer.ref, x.data_ptr(), _DT[x.dtype], y.data_ptr(), _DT[y.dtype], B, workspace.data_ptr(),
        workspace.numel(), s)))
    return y


def q4_linear(x: torch.Tensor, layer: Q4Layer, out_dtype: torch.dtype | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x W^T for x of shape (B, n) or (n,); y has x's dtype unless given."""
    def call(_):
        xx = x.contiguous()
        B = _q4_batch(xx, layer.n, layer.device)
        y = torch.empty((*xx.shape[:-1], layer.m), dtype=out_dtype or x.dtype, device=x.device)
        ws = workspace if workspace is not None else new_q4_workspace(layer, B)
        return q4_linear_into(xx, layer, y, ws)

    return _on_stream(layer.device, stream, call)


def q4_linear_group_into(x: torch.Tensor, layers, ys, workspace: torch.Tensor, stream=None):
    """ys[l] = x W_l^T for 4-bit layers sharing x (a Q4Group, or a list of
    layers); one launch for all of them up to B = 16, and one
    more a layer where the columns are split."""
    group = layers if isinstance(layers, Q4Group) else Q4Group(layers)
    B = _q4_batch(x, group.n, group.device)
    if len(ys) != len(group):
        raise NQError(NQ_ERR_INVALID_ARG, "one output per layer")
    for y, L in zip(ys, group.layers):
        _q4_output(x, B, y, L.m, ys[0].dtype)
    _scratch(workspace, group.device)
    yp = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    _on_stream(group.device, stream, lambda s: _check(lib().nq_q4_linear_fwd_group(
        group.ref, len(group), x.data_ptr(), _DT[x.dtype], yp, _DT[ys[0].dtype], B, workspace.data_ptr(),
        workspace.numel(), s)))
    return ys


def q4_linear_group(x: torch.Tensor, layers, out_dtype: torch.dtype | None = None, stream=None):
    """[x W_l^T] for 4-bit layers sharing x."""
    group = layers if isinstance(layers, Q4Group) else Q4Group(layers)

    def call(_):
        xx = x.contiguous()
        B = _q4_batch(xx, group.n, group.device)
        ys = [torch.empty((*xx.shape[:-1], L.m), dtype=out_dtype or x.dtype, device=x.device) for L in group.layers]
        return q4_linear_group_into(xx, group, ys, new_q4_workspace(group, B))

    return _on_stream(group.device, stream, call)


# ------------------------------------------------------------------ block norms
class BlockNorm:
    """What stands between the linears of two blocks (nq_block_norm): the norm
    behind a block with weight w_post (post=False: none), its gate, the residual
    sum with its scales, and the norm before the next block with weight w_pre
    (pre=False: none).  Weights and the channel gate are (d,) GPU tensors of one
    dtype, fp32, fp16 or bf16; a norm without a weight multiplies by 1."""

    def __init__(self, d: int, act_dtype: torch.dtype = torch.bfloat16, res_dtype: torch.dtype | None = None,
                 w_post: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                 gate: torch.Tensor | None = None, post: bool = True, pre: bool = True, res_scale: float = 1.0,
                 block_scale: float = 1.0, weight_offset: float = 0.0, eps: float = 1e-5):
        given = [t for t in (w_post, w_pre, gate) if t is not None]
        self.d, self.act_dtype, self.res_dtype = d, act_dtype, res_dtype or act_dtype
        self.w_post, self.w_pre, self.gate, self.post, self.pre = w_post, w_pre, gate, post, pre
        self.device = given[0].device if given else None
        dtype = given[0].dtype if given else torch.float32
        for t, name in ((w_post, "w_post"), (w_pre, "w_pre"), (gate, "gate")):
            if t is not None:
                _gpu_tensor(t, name, dtype, (d,), self.device)
        if given and not given[0].is_cuda:
            raise NQError(NQ_ERR_INVALID_ARG, "the weights must be GPU tensors")
        if any(t not in _DT for t in (act_dtype, self.res_dtype, dtype)):
            raise NQError(NQ_ERR_INVALID_ARG, "dtypes must be fp32, fp16 or bf16")
        if (w_post is not None and not post) or (w_pre is not None and not pre):
            raise NQError(NQ_ERR_INVALID_ARG, "a weight for a norm that is left out")
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        self.c = nq_block_norm(d, NQ_NORM_POST * bool(post) | NQ_NORM_PRE * bool(pre), _DT[act_dtype],
                               _DT[self.res_dtype], _DT[dtype], eps, res_scale, block_scale, weight_offset,
                               ptr(w_post), ptr(w_pre), ptr(gate))
        self.ref = ctypes.byref(self.c)

    @staticmethod
    def check(t, name, dtype, shape, device):
        if t is not None:
            _gpu_tensor(t, name, dtype, shape, device)
            return t.data_ptr()
        return None


def _norm_rows(h: torch.Tensor, norm: BlockNorm):
    if h.dim() != 2 or not h.is_cuda or (norm.device is not None and h.device != norm.device):
        raise NQError(NQ_ERR_INVALID_ARG, f"the residual stream must be a (rows, {norm.d}) GPU tensor on the weights' "
                                          "device")
    rows = h.shape[0]
    return rows, (rows, norm.d)


def block_norm(h: torch.Tensor, y: torch.Tensor | None, norm: BlockNorm, gate: torch.Tensor | None = None,
               inplace: bool = False, with_stats: bool = False, stream=None):
    """(h', x) or, with_stats, (h', x, stats): h' = res_scale h + block_scale gate
    post(y), x = pre(h') (None for a norm without `pre`).  h (rows, d) is the
    residual stream, y the block's output, `gate` one gate for each row and
    channel.  inplace writes h' over h; with y None h' is h.  stats (2, rows) is
    what block_norm_backward takes."""
    rows, shape = _norm_rows(h, norm)
    dev, check = h.device, norm.check
    hp, yp = check(h, "h", norm.res_dtype, shape, dev), check(y, "y", norm.act_dtype, shape, dev)
    gp = check(gate, "gate", norm.act_dtype, shape, dev)

    def call(s):
        h_out = h if inplace or y is None else torch.empty_like(h)
        x = torch.empty(shape, dtype=norm.act_dtype, device=dev) if norm.pre else None
        stats = torch.empty((2, rows), dtype=torch.float32, device=dev) if with_stats else None
        _check(lib().nq_block_norm_fwd(norm.ref, rows, hp, yp, gp, h_out.data_ptr(),
                                       x.data_ptr() if norm.pre else None, stats.data_ptr() if with_stats else None,
                                       s))
        return (h_out, x, stats) if with_stats else (h_out, x)

    return _on_stream(dev, stream, call)


def block_norm_backward(dx: torch.Tensor | None, dh: torch.Tensor | None, h: torch.Tensor, y: torch.Tensor | None,
                        stats: torch.Tensor, norm: BlockNorm, gate: torch.Tensor | None = None,
                        inplace: bool = False, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of block_norm from dx and dh, the gradients of x and h' (dh None:
    zero), with h its h' and y, stats and gate as there.  Returns a dict of "dh"
    (written over the given dh with inplace), "dy" (with y) and, where the norm
    has them, "dw_pre", "dw_post" and "dgate" (fp32; for a gate of each row and
    channel its own dtype)."""
    rows, shape = _norm_rows(h, norm)
    dev, check, f32 = h.device, norm.check, torch.float32
    hp, yp = check(h, "h", norm.res_dtype, shape, dev), check(y, "y", norm.act_dtype, shape, dev)
    dxp = check(dx, "dx", norm.act_dtype, shape, dev)
    dhp, gp = check(dh, "dh", norm.res_dtype, shape, dev), check(gate, "gate", norm.act_dtype, shape, dev)
    sp = check(stats, "stats", f32, (2, rows), dev)
    if workspace is not None:
        _scratch(workspace, dev)
    if inplace and dh is None:
        raise NQError(NQ_ERR_INVALID_ARG, "inplace needs dh")

    def call(s):
        out = {"dh": dh if inplace else torch.empty_like(h)}
        if norm.w_pre is not None:
            out["dw_pre"] = torch.empty(norm.d, dtype=f32, device=dev)
        if y is not None and (gate is not None or norm.gate is not None):
            out["dgate"] = torch.empty_like(gate) if gate is not None else torch.empty(norm.d, dtype=f32, device=dev)
        if y is not None and norm.w_post is not None:
            out["dw_post"] = torch.empty(norm.d, dtype=f32, device=dev)
        if y is not None:
            out["dy"] = torch.empty_like(y)
        ptr = lambda k: out[k].data_ptr() if k in out else None  # noqa: E731
        ws = workspace
        if ws is None:
            ws = torch.empty(max(int(lib().nq_block_norm_workspace_bytes(norm.ref, rows)), 256), dtype=torch.uint8,
                             device=dev)
        rows_gate = gate is not None
        _check(lib().nq_block_norm_bwd(norm.ref, rows, dxp, dhp, hp, yp, gp, sp, ptr("dh"), ptr("dy"),
                                       ptr("dgate") if rows_gate else None, ptr("dw_post"), ptr("dw_pre"),
                                       None if rows_gate else ptr("dgate"), ws.data_ptr(), ws.numel(), s))
        return out

    return _on_stream(dev, stream, call)


def bits_per_weight(m: int, n: int, r: int, scale_bits: int = 16) -> float:
    return float(lib().nq_bits_per_weight(m, n, r, scale_bits))


def rank_for_bits(m: int, n: int, bpw: float, scale_bits: int = 16) -> int:
    return int(lib().nq_rank_for_bits(m, n, bpw, scale_bits))


def abi_version() -> int:
    return int(lib().nq_abi_version())
