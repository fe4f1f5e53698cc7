"""Topology-biased graph attention on one GB300 (thin Python binding of libgt).

Every step of the computation runs in the CUDA kernels of libgt.so; this module
only marshals torch tensors into the C ABI declared in include/gt_attn.h (raw
device pointers, sizes, the current CUDA stream) and allocates outputs and
workspace with torch.  There is no CPU path: if libgt.so is missing or cannot
be loaded the calls raise.

Functions (same names as the C entry points):
    gt_spd_build(indptr, indices, n, D)                       -> spd int8 [n][ld]
    gt_bias_attn_fwd(q, k, v, spd, T, scale=None, kv_block=0) -> (o, lse)
    gt_bias_attn_bwd(q, k, v, o, dO, lse, spd, T, scale=None) -> (dq, dk, dv, dT)
    gt_layer_norm_fwd(x, gain, shift, eps)                    -> (y, mean, rstd)
    gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres)          -> (dx, dgain, dshift)
    gt_linear_fwd(x, w, b, act, r)                            -> (y, pre)
    gt_linear_bwd(dy, x, w, pre, act, dx_add)                 -> (dx, dw, db)
The operation follows MegaGraph (abstract: attention scores plus a
topology-aware bias matrix; Fig. 4: blockwise KV streaming with the bias column
slice formed per block) with the Graphormer bias b[h][i][j] = T[h][spd[i][j]].
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

__all__ = [
    "GtError", "load_library", "library_path", "gt_spd_build", "gt_bias_attn_fwd",
    "gt_bias_attn_bwd", "gt_spd_workspace_size", "gt_bias_attn_workspace_size",
    "gt_check_device_status", "gt_status_string", "spd_ld", "GT_F32", "GT_BF16",
    "GT_SPD_AUTO", "GT_SPD_SCAN32", "GT_SPD_SCAN16", "GT_SPD_QUEUE32", "GT_SPD_GLOBAL64",
    "gt_layer_norm_fwd", "gt_layer_norm_bwd", "gt_layer_norm_workspace_size", "gt_linear_fwd", "gt_linear_bwd",
    "gt_linear_fwd_workspace_size", "gt_linear_bwd_workspace_size", "GT_ACT_NONE", "GT_ACT_GELU",
]

GT_F32 = 0
GT_BF16 = 1
# search algorithms of gt_spd_build (include/gt_attn.h)
GT_SPD_AUTO, GT_SPD_SCAN32, GT_SPD_SCAN16, GT_SPD_QUEUE32, GT_SPD_GLOBAL64 = 0, 1, 2, 3, 4
# activations of gt_linear_fwd / gt_linear_bwd
GT_ACT_NONE, GT_ACT_GELU = 0, 1
GT_OK = 0
_STATUS = {0: "GT_OK", -1: "GT_ERR_INVALID_ARG", -2: "GT_ERR_UNSUPPORTED", -3: "GT_ERR_CUDA",
           -4: "GT_ERR_TIMEOUT", -5: "GT_ERR_WORKSPACE"}

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgt.so")
_lock = threading.Lock()
_lib = None


class GtError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        text = _lib.gt_status_string(status).decode() if _lib is not None else ""
        super().__init__(f"{call} returned {_STATUS.get(status, status)}: {text}")


def library_path() -> str:
    return _LIB_PATH


class KernelStat(ctypes.Structure):
    """gt_kernel_stat of the C ABI."""
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


def load_library():
    """Load libgt.so (build it with graph_transformer_attention_gb300.build first)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libgt.so not found at {_LIB_PATH}; run "
                               "`python -m graph_transformer_attention_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(_LIB_PATH)
        P, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                                ctypes.c_float)
        lib.gt_status_string.argtypes = [ctypes.c_int]
        lib.gt_status_string.restype = ctypes.c_char_p
        lib.gt_spd_workspace_size.argtypes = [i32, i64, i32]
        lib.gt_spd_workspace_size.restype = sz
        lib.gt_spd_build.argtypes = [P, P, i32, i64, i32, P, i64, P, sz, P]
        lib.gt_spd_build.restype = ctypes.c_int
        lib.gt_spd_workspace_size_algo.argtypes = [i32, i32, i64, i32]
        lib.gt_spd_workspace_size_algo.restype = sz
        lib.gt_spd_build_algo.argtypes = [i32, P, P, i32, i64, i32, P, i64, P, sz, P]
        lib.gt_spd_build_algo.restype = ctypes.c_int
        lib.gt_bias_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.gt_bias_attn_workspace_size.restype = sz
        lib.gt_bias_attn_fwd_kv_block.argtypes = [i32, i32, i32, i32, i32]
        lib.gt_bias_attn_fwd_kv_block.restype = i32
        lib.gt_bias_attn_fwd_ctas.argtypes = [i32, i32, i32, i32, i32]
        lib.gt_bias_attn_fwd_ctas.restype = i32
        lib.gt_bias_attn_launches.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.gt_bias_attn_launches.restype = ctypes.c_int
        lib.gt_bias_attn_bwd_split.argtypes = [i32, i32, i32, i32, i32]
        lib.gt_bias_attn_bwd_split.restype = i32
        lib.gt_bias_attn_fwd.argtypes = [i32, i32, i32, i32, P, P, P, P, i64, P, i32, f32, i32,
                                         P, P, P, sz, P]
        lib.gt_bias_attn_fwd.restype = ctypes.c_int
        lib.gt_bias_attn_bwd.argtypes = [i32, i32, i32, i32, P, P, P, P, P, P, P, i64, P, i32, f32,
                                         P, P, P, P, P, sz, P]
        lib.gt_bias_attn_bwd.restype = ctypes.c_int
        lib.gt_check_device_status.argtypes = [P]
        lib.gt_check_device_status.restype = ctypes.c_int
        lib.gt_selftest_wait_timeout.argtypes = [i64, P]
        lib.gt_selftest_wait_timeout.restype = ctypes.c_int
        lib.gt_layer_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.gt_layer_workspace_size.restype = sz
        lib.gt_layer_fwd.argtypes = [i32, i32, i32, i32, P, P, P, i64, P, i32, P, P, P, P, P, P, P, sz, P]
        lib.gt_layer_fwd.restype = ctypes.c_int
        lib.gt_layer_bwd.argtypes = [i32, i32, i32, i32, P, P, P, i64, P, i32, P, P, P, P, P, P, P, P, P,
                                     P, sz, P]
        lib.gt_layer_bwd.restype = ctypes.c_int
        lib.gt_bias_attn_fwd_partial.argtypes = [i32, i32, i32, i32, P, P, P, P, i64, P, i32, f32, i32,
                                                 i32, P, P, P]
        lib.gt_bias_attn_fwd_partial.restype = ctypes.c_int
        lib.gt_bias_attn_merge.argtypes = [i32, i32, i32, i32, i32, P, P, P, P, P]
        lib.gt_bias_attn_merge.restype = ctypes.c_int
        lib.gt_layer_norm_fwd.argtypes = [i32, i32, i32, i32, P, i64, P, P, f32, P, i64, P, P, P]
        lib.gt_layer_norm_fwd.restype = ctypes.c_int
        lib.gt_layer_norm_workspace_size.argtypes = [i32, i32]
        lib.gt_layer_norm_workspace_size.restype = sz
        lib.gt_layer_norm_bwd.argtypes = [i32, i32, i32, i32, P, i64, P, i64, P, P, P, P, i64, P, i64, P, P, P, sz, P]
        lib.gt_layer_norm_bwd.restype = ctypes.c_int
        lib.gt_linear_fwd_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.gt_linear_fwd_workspace_size.restype = sz
        lib.gt_linear_fwd.argtypes = [i32, i32, i32, i32, i32, P, i64, P, i64, P, i32, P, i64, P, i64, P, i64,
                                      P, sz, P]
        lib.gt_linear_fwd.restype = ctypes.c_int
        lib.gt_linear_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.gt_linear_bwd_workspace_size.restype = sz
        lib.gt_linear_bwd.argtypes = [i32, i32, i32, i32, i32, P, i64, P, i64, P, i64, P, i64, i32, P, i64, P, i64,
                                      P, i64, P, P, sz, P]
        lib.gt_linear_bwd.restype = ctypes.c_int
        lib.gt_kernel_stats_reset.argtypes = [i32]
        lib.gt_kernel_stats_reset.restype = ctypes.c_int
        lib.gt_kernel_stats_read.argtypes = [ctypes.POINTER(KernelStat), i32, ctypes.POINTER(i32)]
        lib.gt_kernel_stats_read.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(call: str, rc: int):
    if rc != GT_OK:
        raise GtError(call, rc)


def _stream_handle(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GT_F32
    if t.dtype == torch.bfloat16:
        return GT_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("libgt works on CUDA tensors only")
            if not t.is_contiguous():
                raise ValueError("libgt needs contiguous tensors")


def spd_ld(n: int) -> int:
    """Row stride of the SPD matrix: n rounded up to a multiple of 16 bytes."""
    return (n + 15) // 16 * 16


def launches_per_call(dtype: str, h: int, d: int, n: int, kv_block: int = 0, nb: int = 18) -> dict:
    """Number of libgt kernels gt_bias_attn_fwd and gt_bias_attn_bwd launch for
    these sizes on the current device (memsets not counted)."""
    code = GT_F32 if dtype == "f32" else GT_BF16
    fwd, bwd = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("gt_bias_attn_launches",
           load_library().gt_bias_attn_launches(code, n, h, d, nb, kv_block, ctypes.byref(fwd), ctypes.byref(bwd)))
    return {"fwd": int(fwd.value), "bwd": int(bwd.value)}


def gt_status_string(status: int) -> str:
    return load_library().gt_status_string(status).decode()


def gt_spd_workspace_size(n: int, nnz: int, D: int, algo: int = 0) -> int:
    """Workspace bytes of gt_spd_build (0 when `algo` cannot take n vertices here)."""
    return int(load_library().gt_spd_workspace_size_algo(algo, n, nnz, D))


def gt_bias_attn_workspace_size(dtype: int, n: int, h: int, d: int, kv_block: int = 0) -> int:
    return int(load_library().gt_bias_attn_workspace_size(dtype, n, h, d, kv_block))


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def gt_spd_build(indptr: torch.Tensor, indices: torch.Tensor, n: int, D: int,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None, algo: int = 0) -> torch.Tensor:
    """Clipped shortest-path bucket matrix, int8 [n][spd_ld(n)] (columns >= n unspecified).

    `algo` picks the search (GT_SPD_*; 0 = the first that fits the device)."""
    lib = load_library()
    _need_cuda(indptr, indices)
    if indptr.dtype != torch.int64 or indices.dtype != torch.int32:
        raise TypeError("indptr must be int64 and indices int32")
    if out is None:
        out = torch.empty((n, spd_ld(n)), dtype=torch.int8, device=indptr.device)
    if workspace is None:
        need = lib.gt_spd_workspace_size_algo(algo, n, indices.numel(), D)
        if need == 0:
            raise GtError("gt_spd_build", -2)      # the algorithm cannot take n vertices here
        workspace = _workspace(need, indptr.device)
    rc = lib.gt_spd_build_algo(algo, _ptr(indptr), _ptr(indices), n, indices.numel(), D, _ptr(out),
                               out.stride(0), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check("gt_spd_build", rc)
    return out


def gt_bias_attn_fwd(q, k, v, spd, T, scale: float | None = None, kv_block: int = 0,
                     out=None, lse=None, workspace=None, stream=None):
    """Biased attention forward; q, k, v [n][h][d] (fp32 or bf16), spd int8 [n][ld], T fp32 [h][nb]."""
    lib = load_library()
    _need_cuda(q, k, v, spd, T)
    n, h, d = q.shape
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((h, n), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _workspace(lib.gt_bias_attn_workspace_size(dt, n, h, d, kv_block), q.device)
    rc = lib.gt_bias_attn_fwd(dt, n, h, d, _ptr(q), _ptr(k), _ptr(v), _ptr(spd), spd.stride(0),
                              _ptr(T), T.shape[1], float(scale), kv_block, _ptr(out), _ptr(lse),
                              _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check("gt_bias_attn_fwd", rc)
    return out, lse


def gt_bias_attn_fwd_partial(q, k, v, spd, T, kv_begin: int, kv_end: int, scale: float | None = None,
                             o_part=None, lse_part=None, stream=None):
    """Forward over the KV columns [kv_begin, kv_end) only: fp32 o_part [n][h][d]
    (normalised over those columns) and lse_part [h][n]."""
    lib = load_library()
    _need_cuda(q, k, v, spd, T)
    n, h, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o_part is None:
        o_part = torch.empty((n, h, d), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((h, n), dtype=torch.float32, device=q.device)
    _need_cuda(o_part, lse_part)
    rc = lib.gt_bias_attn_fwd_partial(_dtype_code(q), n, h, d, _ptr(q), _ptr(k), _ptr(v), _ptr(spd),
                                      spd.stride(0), _ptr(T), T.shape[1], float(scale), kv_begin, kv_end,
                                      _ptr(o_part), _ptr(lse_part), _stream_handle(stream))
    _check("gt_bias_attn_fwd_partial", rc)
    return o_part, lse_part


def gt_bias_attn_merge(o_parts, lse_parts, dtype=torch.bfloat16, out=None, lse=None, stream=None):
    """Exact merge of partials: o_parts fp32 [p][n][h][d], lse_parts fp32 [p][h][n]."""
    lib = load_library()
    _need_cuda(o_parts, lse_parts)
    nparts, n, h, d = o_parts.shape
    if out is None:
        out = torch.empty((n, h, d), dtype=dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty((h, n), dtype=torch.float32, device=o_parts.device)
    _need_cuda(out, lse)
    rc = lib.gt_bias_attn_merge(_dtype_code(out), n, h, d, nparts, _ptr(o_parts), _ptr(lse_parts),
                                _ptr(out), _ptr(lse), _stream_handle(stream))
    _check("gt_bias_attn_merge", rc)
    return out, lse


def gt_bias_attn_bwd(q, k, v, o, dO, lse, spd, T, scale: float | None = None,
                     dq=None, dk=None, dv=None, dT=None, workspace=None, stream=None):
    """Gradients of sum(o * dO): returns (dq, dk, dv, dT)."""
    lib = load_library()
    _need_cuda(q, k, v, o, dO, lse, spd, T)
    n, h, d = q.shape
    dt = _dtype_code(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dT = torch.empty_like(T) if dT is None else dT
    if workspace is None:
        workspace = _workspace(lib.gt_bias_attn_workspace_size(dt, n, h, d, 0), q.device)
    rc = lib.gt_bias_attn_bwd(dt, n, h, d, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                              _ptr(spd), spd.stride(0), _ptr(T), T.shape[1], float(scale),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dT), _ptr(workspace),
                              workspace.numel(), _stream_handle(stream))
    _check("gt_bias_attn_bwd", rc)
    return dq, dk, dv, dT


LAYER_PARAMS = ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o", "ln2_g", "ln2_b", "w_1", "b_1", "w_2", "b_2")


class _LayerPtrs(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in LAYER_PARAMS]


def _layer_ptrs(tensors: dict) -> _LayerPtrs:
    for name in LAYER_PARAMS:
        t = tensors[name]
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"layer tensor {name} must be contiguous fp32 on the GPU")
    return _LayerPtrs(*[_ptr(tensors[name]) for name in LAYER_PARAMS])


def gt_layer_workspace_size(n: int, h: int = 8, d: int = 8, f: int = 64) -> int:
    return int(load_library().gt_layer_workspace_size(n, h, d, f))


def gt_layer_fwd(x, params: dict, spd, T, workspace=None, stream=None):
    """GT encoder layer forward: y fp32 [n][64] from x fp32 [n][64], and the saved
    tensors of the backward {q, k, v, o (bf16 [n][8][8]), lse}."""
    lib = load_library()
    _need_cuda(x, spd, T)
    n = x.shape[0]
    dev = x.device
    saved = {name: torch.empty((n, 8, 8), dtype=torch.bfloat16, device=dev) for name in ("q", "k", "v", "o")}
    saved["lse"] = torch.empty((8, n), dtype=torch.float32, device=dev)
    y = torch.empty_like(x)
    if workspace is None:
        workspace = _workspace(lib.gt_layer_workspace_size(n, 8, 8, 64), dev)
    w = _layer_ptrs(params)
    rc = lib.gt_layer_fwd(n, 8, 8, 64, _ptr(x), ctypes.byref(w), _ptr(spd), spd.stride(0), _ptr(T), T.shape[1],
                          _ptr(saved["q"]), _ptr(saved["k"]), _ptr(saved["v"]), _ptr(saved["o"]),
                          _ptr(saved["lse"]), _ptr(y), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check("gt_layer_fwd", rc)
    return y, saved


def gt_layer_bwd(x, params: dict, spd, T, saved: dict, dy, workspace=None, stream=None):
    """GT encoder layer backward: (dx, {weight name: gradient}, dT)."""
    lib = load_library()
    _need_cuda(x, spd, T, dy)
    n = x.shape[0]
    dev = x.device
    grads = {name: torch.empty_like(params[name]) for name in LAYER_PARAMS}
    dx = torch.empty_like(x)
    dT = torch.empty_like(T)
    if workspace is None:
        workspace = _workspace(lib.gt_layer_workspace_size(n, 8, 8, 64), dev)
    w = _layer_ptrs(params)
    g = _layer_ptrs(grads)
    rc = lib.gt_layer_bwd(n, 8, 8, 64, _ptr(x), ctypes.byref(w), _ptr(spd), spd.stride(0), _ptr(T), T.shape[1],
                          _ptr(saved["q"]), _ptr(saved["k"]), _ptr(saved["v"]), _ptr(saved["o"]),
                          _ptr(saved["lse"]), _ptr(dy), _ptr(dx), ctypes.byref(g), _ptr(dT), _ptr(workspace),
                          workspace.numel(), _stream_handle(stream))
    _check("gt_layer_bwd", rc)
    return dx, grads, dT


# the handle of a device's current stream and the current device, without the objects around them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _elsewhere(call, first, stream, args):
    """call(*args) on `stream`, or on the device of the tensor `first` where that is not the
    current one.  On another stream than the caller's, results and workspace belong to that
    stream, the caller's tensors stay allocated until its work is done, and the results until the
    caller's stream is done with them."""
    if not first.is_cuda:
        raise ValueError("libgt works on CUDA tensors only")
    if stream is None:
        with torch.cuda.device(first.device):
            return call(*args)
    if stream.device != first.device:
        raise ValueError(f"stream of {stream.device} given for tensors on {first.device}")
    caller = torch.cuda.current_stream(first.device)
    with torch.cuda.stream(stream):
        made = call(*args)
    if caller != stream:
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        for t in made:
            if t is not None:
                t.record_stream(caller)
    return made


def _is_here(t, stream):
    """Whether t's device is the current one and the call goes to its current stream."""
    return stream is None and t.is_cuda and t.device.index == _current_device()


def _matrix(name, t, rows, cols, dtype, device):
    """Leading dimension of a [rows][cols] matrix with unit column stride."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    if rows <= 1:
        return (cols + 7) // 8 * 8       # one row: its stride means nothing
    if ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _vector(name, t, size, device):
    if t.shape != (size,) or t.dtype is not torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous fp32 [{size}] on {device}")
    return t.data_ptr()


def _result(name, t, size, device):
    """(t, address) of an fp32 [size] result: the caller's, or a new one."""
    if t is None:
        t = torch.empty(size, dtype=torch.float32, device=device)
        return t, t.data_ptr()
    return t, _vector(name, t, size, device)


def _matrix_result(name, t, rows, cols, dtype, device):
    """(t, address, leading dimension) of a [rows][cols] result: the caller's, or a new one."""
    if t is None:
        t = torch.empty((rows, cols), dtype=dtype, device=device)
        return t, t.data_ptr(), cols if rows > 1 else (cols + 7) // 8 * 8
    return t, t.data_ptr(), _matrix(name, t, rows, cols, dtype, device)


def _type_code(name, t):
    if t.dtype is torch.float32:
        return GT_F32
    if t.dtype is torch.bfloat16:
        return GT_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


_MOST = 2 ** 31 - 1      # the C calls' sizes are 32-bit, and ctypes would pass a larger one's low bits


def _two_dims(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    rows, cols = t.shape
    if rows > _MOST or cols > _MOST:
        raise ValueError(f"{name} has more than 2^31 - 1 rows or columns")
    return rows, cols


def _room(workspace, need, device):
    """(workspace, address, bytes): the caller's, or a new one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=4096)
def _norm_room(device_index, n, c):
    return int(load_library().gt_layer_norm_workspace_size(n, c))


@functools.lru_cache(maxsize=4096)
def _linear_fwd_room(device_index, dt, m, k, n, aligned):
    return int(load_library().gt_linear_fwd_workspace_size(dt, m, k, n, aligned))


@functools.lru_cache(maxsize=4096)
def _linear_bwd_room(device_index, dt, yt, m, k, n, act, aligned):
    return int(load_library().gt_linear_bwd_workspace_size(dt, yt, m, k, n, act, aligned))


def gt_layer_norm_workspace_size(n: int, c: int) -> int:
    """Workspace bytes of gt_layer_norm_bwd (0 for sizes that are not supported)."""
    if max(n, c) > _MOST:
        return 0
    return int(load_library().gt_layer_norm_workspace_size(n, c))


def gt_linear_fwd_workspace_size(dtype: int, m: int, k: int, n: int, aligned: bool = True) -> int:
    """Workspace bytes of gt_linear_fwd (0: none needed, or sizes that are not supported)."""
    if max(m, k, n) > _MOST:
        return 0
    return int(load_library().gt_linear_fwd_workspace_size(dtype, m, k, n, int(aligned)))


def gt_linear_bwd_workspace_size(dtype: int, ytype: int, m: int, k: int, n: int, act: int = GT_ACT_NONE,
                                 aligned: bool = True) -> int:
    """Workspace bytes of gt_linear_bwd (0: none needed, or sizes that are not supported)."""
    if max(m, k, n) > _MOST:
        return 0
    return int(load_library().gt_linear_bwd_workspace_size(dtype, ytype, m, k, n, act, int(aligned)))


def gt_layer_norm_fwd(x, gain, shift, eps: float = 1e-5, out_dtype=None, out=None, mean=None, rstd=None,
                      stream=None):
    """LayerNorm of the rows of x [n][c] (fp32 or bf16): y [n][c] of out_dtype (default:
    x's type), and fp32 mean [n] and rstd [n] for the backward.  gain, shift fp32 [c]."""
    if not _is_here(x, stream):
        return _elsewhere(gt_layer_norm_fwd, x, stream, (x, gain, shift, eps, out_dtype, out, mean, rstd))
    lib = _lib or load_library()
    n, c = _two_dims("x", x)
    xt, dev = x.dtype, x.device
    yt = out_dtype or (xt if out is None else out.dtype)
    ldx = _matrix("x", x, n, c, xt, dev)
    gp, sp = _vector("gain", gain, c, dev), _vector("shift", shift, c, dev)
    out, yp, ldy = _matrix_result("out", out, n, c, yt, dev)
    mean, mp = _result("mean", mean, n, dev)
    rstd, rp = _result("rstd", rstd, n, dev)
    rc = lib.gt_layer_norm_fwd(_type_code("x", x), _type_code("out", out), n, c, x.data_ptr(), ldx, gp, sp, eps, yp, ldy, mp, rp,
                               _raw_stream(dev.index))
    if rc:
        raise GtError("gt_layer_norm_fwd", rc)
    return out, mean, rstd


def gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=None, dx=None, dgain=None, dshift=None, workspace=None,
                      stream=None):
    """LayerNorm backward from dy = dL/dy and the forward's x, mean, rstd: dx [n][c] of x's
    type (+ dres, the gradient that reaches x around the norm), dgain and dshift fp32 [c]."""
    if not _is_here(x, stream):
        return _elsewhere(gt_layer_norm_bwd, x, stream,
                          (dy, x, gain, mean, rstd, dres, dx, dgain, dshift, workspace))
    lib = _lib or load_library()
    n, c = _two_dims("x", x)
    xt, dev = x.dtype, x.device
    ldx = _matrix("x", x, n, c, xt, dev)
    lddy = _matrix("dy", dy, n, c, dy.dtype, dev)
    gp, mp, rp = _vector("gain", gain, c, dev), _vector("mean", mean, n, dev), _vector("rstd", rstd, n, dev)
    ap, lda = (None, 0) if dres is None else (dres.data_ptr(), _matrix("dres", dres, n, c, xt, dev))
    dx, dxp, lddx = _matrix_result("dx", dx, n, c, xt, dev)
    dgain, dgp = _result("dgain", dgain, c, dev)
    dshift, dsp = _result("dshift", dshift, c, dev)
    workspace, wp, wn = _room(workspace, _norm_room(dev.index, n, c), dev)
    rc = lib.gt_layer_norm_bwd(_type_code("x", x), _type_code("dy", dy), n, c, dy.data_ptr(), lddy, x.data_ptr(), ldx, gp, mp,
                               rp, ap, lda, dxp, lddx, dgp, dsp, wp, wn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_layer_norm_bwd", rc)
    return dx, dgain, dshift


def gt_linear_fwd(x, w, b=None, act: int = GT_ACT_NONE, r=None, out_dtype=None, save_pre: bool = False, out=None,
                  pre=None, workspace=None, stream=None):
    """y = act(x w + b) + r: x [m][k] and w [k][n] of one type (fp32 or bf16), b fp32 [n], r
    [m][n] of y's type.  Returns (y, pre): y of out_dtype (default: r's type, else x's; fp32
    for fp32 products), pre = x w + b of x's type with save_pre (or given to write to), else None."""
    if not _is_here(x, stream):
        return _elsewhere(gt_linear_fwd, x, stream, (x, w, b, act, r, out_dtype, save_pre, out, pre, workspace))
    lib = _lib or load_library()
    m, k = _two_dims("x", x)
    n = _two_dims("w", w)[1]
    xt, dev = x.dtype, x.device
    dt = _type_code("x", x)
    ldx, ldw = _matrix("x", x, m, k, xt, dev), _matrix("w", w, k, n, xt, dev)
    yt = out_dtype or (out.dtype if out is not None else r.dtype if r is not None else xt)
    bp = None if b is None else _vector("b", b, n, dev)
    rp, ldr = (None, 0) if r is None else (r.data_ptr(), _matrix("r", r, m, n, yt, dev))
    out, yp, ldy = _matrix_result("out", out, m, n, yt, dev)
    pp, ldp = None, 0
    if save_pre or pre is not None:
        pre, pp, ldp = _matrix_result("pre", pre, m, n, xt, dev)
    xp, wp = x.data_ptr(), w.data_ptr()
    # rows of whole 16 bytes
    ex, ey = x.element_size(), out.element_size()
    aligned = (xp | wp | yp | (rp or 0) | (pp or 0) | (ldx | ldw | ldp) * ex | (ldy | ldr) * ey) % 16 == 0
    workspace, sp, sn = _room(workspace, _linear_fwd_room(dev.index, dt, m, k, n, aligned), dev)
    rc = lib.gt_linear_fwd(dt, _type_code("out", out), m, k, n, xp, ldx, wp, ldw, bp, act, rp, ldr, yp, ldy, pp,
                           ldp, sp, sn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_linear_fwd", rc)
    return out, pre


def gt_linear_bwd(dy, x, w, pre=None, act: int = GT_ACT_NONE, dx_add=None, need_dx: bool = True,
                  need_dw: bool = True, need_db: bool = True, dx=None, dw=None, db=None, workspace=None,
                  stream=None):
    """Backward of gt_linear_fwd from dy = dL/dy [m][n]: (dx [m][k], dw [k][n], db fp32 [n]), dx
    and dw of x's type, None for those not needed.  pre: the forward's, with GELU.  dx_add
    [m][k]: a gradient that reaches x another way, added to dx.  x may be None where dw is not
    needed, w where dx is not (one of the two gives the sizes and the type)."""
    if not _is_here(dy, stream):
        return _elsewhere(gt_linear_bwd, dy, stream, (dy, x, w, pre, act, dx_add, need_dx, need_dw, need_db, dx, dw, db,
                                                      workspace))
    lib = _lib or load_library()
    need_dx, need_dw = need_dx or dx is not None, need_dw or dw is not None
    if (x is None and (need_dw or w is None)) or (w is None and need_dx):
        raise ValueError("x may be None only where dw is not needed, w where dx is not, and not both")
    m, n = _two_dims("dy", dy)
    k = _two_dims("w", w)[0] if x is None else _two_dims("x", x)[1]
    given = w if x is None else x
    xt, dev = given.dtype, dy.device
    dt, yt = _type_code("w" if x is None else "x", given), _type_code("dy", dy)
    xp, ldx = (None, 0) if x is None else (x.data_ptr(), _matrix("x", x, m, k, xt, dev))
    wp, ldw = (None, 0) if w is None else (w.data_ptr(), _matrix("w", w, k, n, xt, dev))
    lddy = _matrix("dy", dy, m, n, dy.dtype, dev)
    pp, ldp = (None, 0) if pre is None else (pre.data_ptr(), _matrix("pre", pre, m, n, xt, dev))
    ap, lda = (None, 0) if dx_add is None else (dx_add.data_ptr(), _matrix("dx_add", dx_add, m, k, xt, dev))
    dxp, lddx, dwp, lddw, dbp = None, 0, None, 0, None
    if need_dx:
        dx, dxp, lddx = _matrix_result("dx", dx, m, k, xt, dev)
    if need_dw:
        dw, dwp, lddw = _matrix_result("dw", dw, k, n, xt, dev)
    if need_db or db is not None:
        db, dbp = _result("db", db, n, dev)
    dyp = dy.data_ptr()
    aligned = ((xp or 0) | (wp or 0) | dyp | (pp or 0) | (ap or 0) | (dxp or 0) | (dwp or 0) | lddy * dy.element_size() |
               (ldx | ldw | ldp | lda | lddx | lddw) * given.element_size()) % 16 == 0
    workspace, sp, sn = _room(workspace, _linear_bwd_room(dev.index, dt, yt, m, k, n, act, aligned), dev)
    rc = lib.gt_linear_bwd(dt, yt, m, k, n, dyp, lddy, xp, ldx, wp, ldw, pp, ldp, act, ap, lda, dxp, lddx, dwp, lddw,
                           dbp, sp, sn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_linear_bwd", rc)
    return dx, dw, db


def gt_check_device_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel gave up a bounded wait."""
    _check("gt_check_device_status", load_library().gt_check_device_status(_stream_handle(stream)))


def gt_selftest_wait_timeout(limit_ns: int = 50_000_000, stream=None) -> None:
    """Launch the library's bounded-wait self-test: a wait that nothing ends, which
    gives up after limit_ns; the next gt_check_device_status reports GT_ERR_TIMEOUT."""
    _check("gt_selftest_wait_timeout",
           load_library().gt_selftest_wait_timeout(int(limit_ns), _stream_handle(stream)))


def gt_kernel_stats_reset(timing: bool = False) -> None:
    """Clear the library's launch table; with timing, bracket every launch with
    CUDA events on its stream from now on."""
    _check("gt_kernel_stats_reset", load_library().gt_kernel_stats_reset(1 if timing else 0))


def gt_kernel_stats() -> dict:
    """{kernel name: (launches, total device ms or -1 without timing)} since the
    last reset, in first-launch order."""
    lib = load_library()
    count = ctypes.c_int32(0)
    _check("gt_kernel_stats_read", lib.gt_kernel_stats_read(None, 0, ctypes.byref(count)))
    arr = (KernelStat * max(1, count.value))()
    _check("gt_kernel_stats_read", lib.gt_kernel_stats_read(arr, count.value, ctypes.byref(count)))
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms))
            for i in range(count.value)}
