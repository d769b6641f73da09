"""Python binding of libnq: linear layers with a low-rank binary-factorised weight
W_hat = diag(s1) U diag(g) V^T diag(s2) on MI355X, and what stands beside them in a
model: linears with 4-bit weights (q4_*), the norms between blocks (block_norm), the
norms and rotation of heads (head_norm), a paged cache of keys and values (kv_write,
kv_read) and one token's attention over it (kv_attention).

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
NQ_HEAD_NORM, NQ_HEAD_INTERLEAVED, NQ_HEAD_MAX_AXES = 1, 2, 4  # head norms (include/nq.h)
KV_KINDS = {"bf16": 0, "int8": 1, "int4": 2}  # how a cache holds its values (include/nq.h)
_INT32_MAX = 2 ** 31 - 1  # more than a call's tokens: ctypes would cut a wider whole number to its lower bits
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


class nq_kv_cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("kind", ctypes.c_int32), ("data", ctypes.c_void_p)]


class nq_head_norm(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("flags", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("rot", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * NQ_HEAD_MAX_AXES), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p)]


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
    K, H, c_long = ctypes.POINTER(nq_kv_cache), ctypes.POINTER(nq_head_norm), ctypes.c_int64
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
        "nq_kv_page_bytes": (c_size, [c_int, c_int, c_int, c_int]),
        "nq_kv_write": (c_int, [K, c_int, vp, c_long, vp, c_long, c_int, vp, vp]),
        "nq_kv_read": (c_int, [K, c_int, vp, vp, vp, c_int, vp]),
        "nq_kv_attention_workspace_bytes": (c_size, [K]),
        "nq_kv_attention": (c_int, [K, c_int, vp, c_int, c_int, vp, c_int, vp, c_int, c_int, ctypes.c_float, vp, c_int,
                                    vp, c_size, vp]),
        "nq_head_norm_fwd": (c_int, [H, c_int, vp, c_long, c_int, vp, c_long, c_int, vp, vp, vp, vp]),
        "nq_head_norm_kv_write": (c_int, [H, c_int, vp, c_long, c_int, vp, c_long, vp, c_long, vp, K, vp, vp, vp]),
        "nq_head_norm_workspace_bytes": (c_size, [H, c_int]),
        "nq_head_norm_bwd": (c_int, [H, c_int, vp, vp, vp, c_long, c_int, vp, c_long, c_int, vp, vp, vp, vp, vp, vp,
                                     c_size, vp]),
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


# ------------------------------------------------------------------ cache of keys and values
class KvCache:
    """Keys and values of many sequences in `pages` pages of `page` slots (a multiple
    of 16), a slot holding one token's `heads` heads of `head_dim` (64, 96, 128, 192 or
    256) channels, as bf16 ("bf16") or as whole numbers of 8 ("int8", one scale for each
    token and head) or 4 bits ("int4", one for 32 channels of it): nq_kv_cache.  `data`
    (pages, bytes of a page) is uint8 in the kernels' own order; `into` gives that memory."""

    def __init__(self, pages: int, heads: int, head_dim: int, page: int = 64, kind: str = "bf16", device="cuda",
                 into: torch.Tensor | None = None):
        if kind not in KV_KINDS:
            raise NQError(NQ_ERR_INVALID_ARG, f"kind must be one of {', '.join(KV_KINDS)}")
        nbytes = int(lib().nq_kv_page_bytes(heads, head_dim, page, KV_KINDS[kind]))
        if nbytes == 0 or not 1 <= pages <= 1 << 24:
            raise NQError(NQ_ERR_INVALID_ARG, f"invalid cache pages={pages} heads={heads} head_dim={head_dim} page={page}")
        if into is not None:
            if into.dtype != torch.uint8 or into.shape != (pages, nbytes) or not into.is_cuda or not into.is_contiguous():
                raise NQError(NQ_ERR_INVALID_ARG, f"into must be a contiguous uint8 GPU tensor of shape {(pages, nbytes)}")
        self.data = into if into is not None else torch.empty((pages, nbytes), dtype=torch.uint8, device=device)
        self.pages, self.heads, self.head_dim, self.page, self.kind = pages, heads, head_dim, page, kind
        self.page_bytes, self.device = nbytes, self.data.device
        self.c = nq_kv_cache(pages, heads, head_dim, page, KV_KINDS[kind], self.data.data_ptr())
        self.ref = ctypes.byref(self.c)


def _like(t: torch.Tensor, dtype=None) -> torch.Tensor:
    """A contiguous tensor of t's shape; 0.5 us less than naming shape, type and device."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _head_rows(t: torch.Tensor, name: str, dtype, heads, D: int, device) -> int:
    """Elements between the rows of a (tokens, heads, D) tensor whose tokens are
    contiguous: a tensor of its own or a part of a wider linear's output."""
    shape = t.shape
    if t.dtype == dtype and t.device == device and len(shape) == 3 and shape[2] == D and (heads is None or
                                                                                         shape[1] == heads):
        if t.is_contiguous():
            return shape[1] * D
        s = t.stride()
        if s[2] == 1 and (s[1] == D or shape[1] == 1):
            return s[0]
    raise NQError(NQ_ERR_INVALID_ARG, f"{name} must be a {dtype} tensor (tokens, {'heads' if heads is None else heads}, "
                                      f"{D}) on {device}, each token contiguous (got {t.dtype} {tuple(shape)} on {t.device})")


def _kv_slots(slots: torch.Tensor, tokens: int, device) -> None:
    if slots.dtype != torch.int64 or slots.shape != (tokens,) or slots.device != device or not slots.is_contiguous():
        raise NQError(NQ_ERR_INVALID_ARG, f"slots must be a contiguous int64 tensor of shape ({tokens},) on {device}")


def kv_write(k: torch.Tensor, v: torch.Tensor, cache: KvCache, slots: torch.Tensor, stream=None) -> None:
    """Writes tokens' keys and values (tokens, heads, head_dim; bf16 or fp32, rows may be
    parts of wider ones) to their slots (int64; place s % page of page s // page; a slot
    outside the cache, a negative one say, is left out)."""
    if k.dtype not in _ACT:
        raise NQError(NQ_ERR_INVALID_ARG, "k and v must be bf16 or fp32")
    ks = _head_rows(k, "k", k.dtype, cache.heads, cache.head_dim, cache.device)
    vs = _head_rows(v, "v", k.dtype, cache.heads, cache.head_dim, cache.device)
    tokens = k.shape[0]
    if v.shape[0] != tokens:
        raise NQError(NQ_ERR_INVALID_ARG, f"{tokens} keys and {v.shape[0]} values")
    _kv_slots(slots, tokens, cache.device)
    _on_stream(cache.device, stream, lambda s: _check(lib().nq_kv_write(
        cache.ref, tokens, k.data_ptr(), ks, v.data_ptr(), vs, _DT[k.dtype], slots.data_ptr(), s)))


def kv_read(cache: KvCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """(k, v), (tokens, heads, head_dim) each: the values that the slots hold; zeros for
    a slot outside the cache."""
    if dtype not in _ACT:
        raise NQError(NQ_ERR_INVALID_ARG, "dtype must be bf16 or fp32")
    tokens = slots.shape[0] if slots.dim() == 1 else -1
    _kv_slots(slots, tokens, cache.device)

    def call(s):
        k = cache.data.new_empty((tokens, cache.heads, cache.head_dim), dtype=dtype)
        v = _like(k)
        _check(lib().nq_kv_read(cache.ref, tokens, slots.data_ptr(), k.data_ptr(), v.data_ptr(), _DT[dtype], s))
        return k, v

    return _on_stream(cache.device, stream, call)


def kv_attention_workspace_bytes(cache: KvCache) -> int:
    """Workspace of kv_attention over this cache, for any batch."""
    return int(lib().nq_kv_attention_workspace_bytes(cache.ref))


def new_kv_workspace(B: int, q_heads: int, cache: KvCache) -> torch.Tensor:
    """A workspace for kv_attention of B sequences and q_heads heads (its size depends on
    the cache alone)."""
    return torch.empty(kv_attention_workspace_bytes(cache), dtype=torch.uint8, device=cache.device)


def kv_attention_into(q: torch.Tensor, cache: KvCache, table: torch.Tensor, lengths: torch.Tensor, y: torch.Tensor,
                      workspace: torch.Tensor, scale: float | None = None, window: int = 0, max_length: int = 0,
                      stream=None) -> torch.Tensor:
    """kv_attention into caller buffers (safe to capture in a graph: lengths and table are
    read by the kernels)."""
    dev = cache.device
    B, q_heads = (q.shape[0], q.shape[1]) if q.dim() == 3 else (-1, -1)
    if q.dtype not in _ACT or y.dtype not in _ACT:
        raise NQError(NQ_ERR_INVALID_ARG, "q and y must be bf16 or fp32")
    _gpu_tensor(q, "q", q.dtype, (B, q_heads, cache.head_dim), dev)
    _gpu_tensor(y, "y", y.dtype, q.shape, dev)
    _gpu_tensor(lengths, "lengths", torch.int32, (B,), dev)
    if table.dim() != 2:
        raise NQError(NQ_ERR_INVALID_ARG, "table must be (sequences, pages)")
    _gpu_tensor(table, "table", torch.int32, (B, table.shape[1]), dev)
    _scratch(workspace, dev)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    if window < 0 or max_length < 0:
        raise NQError(NQ_ERR_INVALID_ARG, f"max_length {max_length} or window {window} below zero")
    _on_stream(dev, stream, lambda s: _check(lib().nq_kv_attention(
        cache.ref, B, q.data_ptr(), _DT[q.dtype], q_heads, table.data_ptr(), table.shape[1], lengths.data_ptr(),
        min(max_length, _INT32_MAX), min(window, _INT32_MAX), scale, y.data_ptr(), _DT[y.dtype], workspace.data_ptr(), workspace.numel(), s)))
    return y


def kv_attention(q: torch.Tensor, cache: KvCache, table: torch.Tensor, lengths: torch.Tensor,
                 scale: float | None = None, window: int = 0, max_length: int = 0,
                 out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Attention of one new token a sequence: q (B, q_heads, head_dim) bf16 or fp32, over
    the last `window` (0: all) of lengths[b] tokens (int32; the new one, already written,
    among them), whose token t lies in slot t % page of page table[b, t // page] (int32).
    Query head h reads key head h // (q_heads // heads); scale is head_dim ** -0.5 unless
    given.  Returns (B, q_heads, head_dim) of q's dtype unless given; zeros for a length
    of 0, NaN for one above max_length (what the host knows of the lengths; 0: what the
    table holds) or a page outside the cache."""
    def call(_):
        ws = workspace if workspace is not None else new_kv_workspace(0, 0, cache)  # of any batch; q is checked below
        return kv_attention_into(q, cache, table, lengths, _like(q, out_dtype), ws, scale, window,
                                 max_length)

    return _on_stream(cache.device, stream, call)


# ------------------------------------------------------------------ head norms
class HeadNorm:
    """Norm of each head of queries and keys with weights w_q and w_k ((head_dim,) GPU
    tensors of one dtype, fp32, fp16 or bf16, or None for 1; norm=False: no norm), and
    the rotation of its first 2 * len(inv_freq) channels by position * inv_freq (fp64, or
    anything that converts to it; None: no rotation), pairs (i, i + rot / 2) or, interleaved,
    (2i, 2i + 1).  sections: how many of the pairs go by each axis of the positions, in
    order (None: one axis).  See nq_head_norm in include/nq.h."""

    def __init__(self, head_dim: int, act_dtype: torch.dtype = torch.bfloat16, w_q: torch.Tensor | None = None,
                 w_k: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                 sections=None, norm: bool = True, weight_offset: float = 0.0, eps: float = 1e-6):
        given = [t for t in (w_q, w_k) if t is not None]
        self.head_dim, self.act_dtype, self.w_q, self.w_k, self.norm = head_dim, act_dtype, w_q, w_k, norm
        dtype = given[0].dtype if given else torch.float32
        self.device = given[0].device if given else inv_freq.device if inv_freq is not None else None
        for t, name in ((w_q, "w_q"), (w_k, "w_k")):
            if t is not None:
                _gpu_tensor(t, name, dtype, (head_dim,), self.device)
        if act_dtype not in _ACT or dtype not in _DT:
            raise NQError(NQ_ERR_INVALID_ARG, "heads must be bf16 or fp32, weights fp32, fp16 or bf16")
        if given and not norm:
            raise NQError(NQ_ERR_INVALID_ARG, "a weight for a norm that is left out")
        if self.device is not None and self.device.type != "cuda":
            raise NQError(NQ_ERR_INVALID_ARG, "the weights and inv_freq must be GPU tensors")
        if inv_freq is not None and (inv_freq.dim() != 1 or inv_freq.device != self.device):
            raise NQError(NQ_ERR_INVALID_ARG, f"inv_freq must be one row on {self.device}")
        self.inv_freq = inv_freq.double().contiguous() if inv_freq is not None else None
        pairs = inv_freq.shape[0] if inv_freq is not None else 0
        self.sections = tuple(int(n) for n in sections) if sections is not None else (pairs,)
        self.axes = len(self.sections)
        if not 1 <= self.axes <= NQ_HEAD_MAX_AXES or sum(self.sections) != pairs or min(self.sections) < 0:
            raise NQError(NQ_ERR_INVALID_ARG, f"sections {self.sections} for {pairs} pairs and up to {NQ_HEAD_MAX_AXES} axes")
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        self.c = nq_head_norm(head_dim, NQ_HEAD_NORM * bool(norm) | NQ_HEAD_INTERLEAVED * bool(interleaved),
                              _DT[act_dtype], _DT[dtype], 2 * pairs, self.axes,
                              (ctypes.c_int32 * NQ_HEAD_MAX_AXES)(*self.sections), eps, weight_offset, ptr(w_q),
                              ptr(w_k), ptr(self.inv_freq))
        self.ref = ctypes.byref(self.c)

    def check(self, q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None):
        """(device, tokens, heads and row strides of q and k, address of the positions)."""
        some = q if q is not None else k
        if some is None or not some.is_cuda or (self.device is not None and some.device != self.device):
            raise NQError(NQ_ERR_INVALID_ARG, "q or k must be given, on the weights' device")
        dev, tokens = some.device, some.shape[0] if some.dim() == 3 else -1
        qs = _head_rows(q, "q", self.act_dtype, None, self.head_dim, dev) if q is not None else 0
        ks = _head_rows(k, "k", self.act_dtype, None, self.head_dim, dev) if k is not None else 0
        if k is not None and k.shape[0] != tokens:
            raise NQError(NQ_ERR_INVALID_ARG, f"q of {tokens} tokens, k of {k.shape[0]}")
        pp = None
        if self.inv_freq is not None:
            shape = positions.shape if positions is not None else None
            if shape is None or positions.dtype != torch.int64 or positions.device != dev or \
                    not positions.is_contiguous() or (shape != (self.axes, tokens) and
                                                      not (self.axes == 1 and shape == (tokens,))):
                raise NQError(NQ_ERR_INVALID_ARG, f"positions must be a contiguous int64 tensor of shape ({self.axes}, "
                                                  f"{tokens}) on {dev}")
            pp = positions.data_ptr()
        return dev, tokens, q.shape[1] if q is not None else 0, qs, k.shape[1] if k is not None else 0, ks, pp


def head_norm(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None, norm: HeadNorm,
              inplace: bool = False, stream=None):
    """(q', k'): norm and rotation of the heads of q and k, (tokens, heads, head_dim) each
    (either may be None; rows may be parts of wider ones), at positions (tokens,) or
    (axes, tokens) int64.  inplace writes over contiguous q and k."""
    dev, tokens, qh, qs, kh, ks, pp = norm.check(q, k, positions)
    if inplace and not all(t is None or t.is_contiguous() for t in (q, k)):
        raise NQError(NQ_ERR_INVALID_ARG, "inplace needs contiguous q and k")

    def call(s):
        qo = q if q is None or inplace else _like(q)
        ko = k if k is None or inplace else _like(k)
        _check(lib().nq_head_norm_fwd(norm.ref, tokens, q.data_ptr() if qh else None, qs, qh,
                                      k.data_ptr() if kh else None, ks, kh, pp, qo.data_ptr() if qh else None,
                                      ko.data_ptr() if kh else None, s))
        return qo, ko

    return _on_stream(dev, stream, call)


def head_norm_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None, norm: HeadNorm,
                    cache: KvCache, slots: torch.Tensor, stream=None) -> torch.Tensor:
    """q' of head_norm, with k' and v written to the cache's slots in the same launch: what
    head_norm and then kv_write(k', v, cache, slots) leave there, bit for bit."""
    dev, tokens, qh, qs, kh, ks, pp = norm.check(q, k, positions)
    vs = _head_rows(v, "v", norm.act_dtype, kh, norm.head_dim, dev)
    if cache.device != dev or cache.heads != kh or v.shape[0] != tokens:
        raise NQError(NQ_ERR_INVALID_ARG, f"k and v must have the cache's {cache.heads} heads, on {cache.device}, and "
                                          f"{tokens} tokens")
    _kv_slots(slots, tokens, dev)

    def call(s):
        qo = _like(q)
        _check(lib().nq_head_norm_kv_write(norm.ref, tokens, q.data_ptr(), qs, qh, k.data_ptr(), ks, v.data_ptr(), vs,
                                           pp, cache.ref, slots.data_ptr(), qo.data_ptr(), s))
        return qo

    return _on_stream(dev, stream, call)


def head_norm_backward(dq: torch.Tensor | None, dk: torch.Tensor | None, q: torch.Tensor | None,
                       k: torch.Tensor | None, positions: torch.Tensor | None, norm: HeadNorm, inplace: bool = False,
                       workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of head_norm from dq and dk, those of q' and k' (contiguous), with q, k and
    positions as there.  Returns a dict of "dq" and "dk" (written over the given ones with
    inplace) for the q and k that are given and, where the norm has the weight, "dw_q" and
    "dw_k" (fp32, sums over tokens and heads)."""
    dev, tokens, qh, qs, kh, ks, pp = norm.check(q, k, positions)
    if (dq is None) != (q is None) or (dk is None) != (k is None):
        raise NQError(NQ_ERR_INVALID_ARG, "a gradient for each of q and k that is given")
    for d, t, name in ((dq, q, "dq"), (dk, k, "dk")):
        if t is not None:
            _gpu_tensor(d, name, norm.act_dtype, t.shape, dev)
    if workspace is not None:
        _scratch(workspace, dev)
    some = q if q is not None else k

    def call(s):
        out = {}
        for name, d in (("dq", dq), ("dk", dk)):
            if d is not None:
                out[name] = d if inplace else _like(d)
        for name, w, t in (("dw_q", norm.w_q, q), ("dw_k", norm.w_k, k)):
            if w is not None and t is not None:
                out[name] = _like(w, torch.float32)
        ptr = lambda key: out[key].data_ptr() if key in out else None  # noqa: E731
        ws = workspace
        if ws is None:
            ws = some.new_empty(max(int(lib().nq_head_norm_workspace_bytes(norm.ref, tokens)), 256), dtype=torch.uint8)
        _check(lib().nq_head_norm_bwd(norm.ref, tokens, dq.data_ptr() if qh else None, dk.data_ptr() if kh else None,
                                      q.data_ptr() if qh else None, qs, qh, k.data_ptr() if kh else None, ks, kh, pp,
                                      ptr("dq"), ptr("dk"), ptr("dw_q"), ptr("dw_k"), ws.data_ptr(), ws.numel(), s))
        return out

    return _on_stream(dev, stream, call)


def bits_per_weight(m: int, n: int, r: int, scale_bits: int = 16) -> float:
    return float(lib().nq_bits_per_weight(m, n, r, scale_bits))


def rank_for_bits(m: int, n: int, bpw: float, scale_bits: int = 16) -> int:
    return int(lib().nq_rank_for_bits(m, n, bpw, scale_bits))


def abi_version() -> int:
    return int(lib().nq_abi_version())
