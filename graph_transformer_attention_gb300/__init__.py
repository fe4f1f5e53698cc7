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
    gt_qk_norm_fwd(q, k, gain_q, gain_k, freq, pos_q, pos_k)  -> (yq, yk)
    gt_qk_norm_bwd(dyq, dyk, q, k, gain_q, gain_k, freq, ..)  -> (dq, dk, dgain_q, dgain_k)
    gt_cross_attn_fwd(q, k, v, q_off, kv_off, key_mask)       -> (o, lse)
    gt_cross_attn_bwd(q, k, v, o, dO, lse, q_off, kv_off, ..) -> (dq, dk, dv)
    gt_grad_clip(grads, max_norm, out)                        -> norm
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
    "gt_cross_attn_fwd", "gt_cross_attn_bwd", "gt_cross_attn_workspace_size", "gt_qk_norm_fwd", "gt_qk_norm_bwd",
    "gt_qk_norm_workspace_size", "GT_ROT_HALVES", "GT_ROT_PAIRS", "gt_grad_clip", "gt_tensor_list",
    "gt_grad_clip_workspace_size",
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
        lib.gt_cross_attn_workspace_size.argtypes = [i32] * 9
        lib.gt_cross_attn_workspace_size.restype = sz
        view = [P, i64, i64]
        lib.gt_cross_attn_fwd.argtypes = [i32] * 7 + view * 3 + [P, P, P, f32] + view + [P, P, sz, P]
        lib.gt_cross_attn_fwd.restype = ctypes.c_int
        lib.gt_cross_attn_bwd.argtypes = [i32] * 7 + view * 5 + [P, P, P, P, f32] + view * 3 + [P, sz, P]
        lib.gt_cross_attn_bwd.restype = ctypes.c_int
        lib.gt_qk_norm_fwd.argtypes = [i32, i32, i32, f32, P, i32, i32] + ([i32, i32] + view + [P, P] + view) * 2 + [P]
        lib.gt_qk_norm_fwd.restype = ctypes.c_int
        lib.gt_qk_norm_workspace_size.argtypes = [i32]
        lib.gt_qk_norm_workspace_size.restype = sz
        lib.gt_qk_norm_bwd.argtypes = ([i32, i32, i32, f32, P, i32, i32] +
                                       ([i32, i32] + view * 2 + [P, P] + view + [P]) * 2 + [P, sz, P])
        lib.gt_qk_norm_bwd.restype = ctypes.c_int
        lib.gt_grad_clip_workspace_size.argtypes = [i32]
        lib.gt_grad_clip_workspace_size.restype = sz
        lib.gt_grad_clip.argtypes = [P, i32, f32, P, P, sz, P]
        lib.gt_grad_clip.restype = ctypes.c_int
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


GT_ROT_HALVES = 0
GT_ROT_PAIRS = 1


def _heads(name, t, rows, heads, d, dtype, device, result=False):
    """(address, row stride, head stride) of a [rows][heads][d] tensor with contiguous channels."""
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name} must be [{rows}][{heads}][{d}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")
    ld, hd, unit = t.stride()
    if unit != 1 and d > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    # the stride of a single head or row means nothing
    if heads == 1:
        hd = (d + 7) // 8 * 8
    if rows == 1:
        ld = (heads * hd + 7) // 8 * 8
    if result and not ((heads == 1 or hd >= d) and (rows == 1 or ld >= (heads - 1) * hd + d) or
                       (rows == 1 or ld >= d) and (heads == 1 or hd >= (rows - 1) * ld + d)):
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), ld, hd


def _heads_result(name, t, rows, heads, d, dtype, device):
    """(t, (address, row stride, head stride)) of a [rows][heads][d] result: the caller's, or a new one."""
    if t is None:
        t = torch.empty((rows, heads, d), dtype=dtype, device=device)
    return t, _heads(name, t, rows, heads, d, dtype, device, result=True)


def _three_dims(name, t):
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions, got {t.dim()}")
    if max(t.shape) > _MOST:
        raise ValueError(f"{name} has more than 2^31 - 1 rows, heads or channels")
    return t.shape


def _ints(name, t, size, device):
    if t.shape != (size,) or t.dtype is not torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [{size}] on {device}")
    return t.data_ptr()


def _sequences(q_off, kv_off, nk, key_mask, device):
    """(batch, addresses of the offsets and of the mask)"""
    if (q_off is None) != (kv_off is None):
        raise ValueError("q_off and kv_off belong together")
    batch, qp, kp, mp = 1, None, None, None
    if q_off is not None:
        batch = q_off.numel() - 1
        if batch < 1:
            raise ValueError("q_off must have at least 2 values")
        qp, kp = _ints("q_off", q_off, batch + 1, device), _ints("kv_off", kv_off, batch + 1, device)
    if key_mask is not None:
        if (key_mask.shape != (nk,) or key_mask.dtype not in (torch.bool, torch.uint8) or key_mask.device != device or
                not key_mask.is_contiguous()):
            raise ValueError(f"key_mask must be contiguous bool or uint8 [{nk}] on {device}")
        mp = key_mask.data_ptr()
    return batch, qp, kp, mp


def _in_place(*views):
    """Whether rows of bf16 are read without a copy: bases and strides of whole 16 bytes, no stride of 0."""
    bits = 0
    for p, ld, hd in views:
        if ld == 0 or hd == 0:
            return False
        bits |= p | 2 * ld | 2 * hd
    return bits % 16 == 0


@functools.lru_cache(maxsize=4096)
def _cross_room(device_index, dt, nq, nk, h, hk, d, batch, backward, aligned):
    return int(load_library().gt_cross_attn_workspace_size(dt, nq, nk, h, hk, d, batch, backward, aligned))


def gt_cross_attn_workspace_size(dtype: int, nq: int, nk: int, h: int, hk: int, d: int, batch: int = 1,
                                 backward: bool = False, aligned: bool = True) -> int:
    """Workspace bytes of gt_cross_attn_fwd or, with backward, of gt_cross_attn_bwd (0: none needed, or sizes
    that are not supported).  aligned: all bf16 inputs have bases and strides of whole 16 bytes."""
    if max(nq, nk, h, hk, d, batch) > _MOST:
        return 0
    return int(load_library().gt_cross_attn_workspace_size(dtype, nq, nk, h, hk, d, batch, int(backward), int(aligned)))


def _lse_of(lse, h, nq, device):
    if lse.shape != (h, nq) or lse.dtype is not torch.float32 or lse.device != device or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous fp32 [{h}][{nq}] on {device}")
    return lse.data_ptr()


def gt_cross_attn_fwd(q, k, v, q_off=None, kv_off=None, key_mask=None, scale: float | None = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Cross attention forward: o [nq][h][d] and lse fp32 [h][nq] of queries q [nq][h][d] over k and v [nk][hk][d]
    (fp32 or bf16; query head j reads key head j / (h / hk); rows and heads may be strided).

    q_off, kv_off int32 [batch + 1]: packed sequences, each with its own keys (default: one sequence).  key_mask bool
    or uint8 [nk]: keys with 0 are not seen.  scale: 1 / sqrt(d) by default.  A query that sees no key has o = 0 and
    lse = -infinity; rows outside the sequences are not written."""
    if not _is_here(q, stream):
        return _elsewhere(gt_cross_attn_fwd, q, stream, (q, k, v, q_off, kv_off, key_mask, scale, out, lse, workspace))
    lib = _lib or load_library()
    nq, h, d = _three_dims("q", q)
    nk, hk, _ = _three_dims("k", k)
    xt, dev, dt = q.dtype, q.device, _type_code("q", q)
    qv, kv, vv = _heads("q", q, nq, h, d, xt, dev), _heads("k", k, nk, hk, d, xt, dev), _heads("v", v, nk, hk, d, xt, dev)
    batch, qp, kp, mp = _sequences(q_off, kv_off, nk, key_mask, dev)
    out, ov = _heads_result("out", out, nq, h, d, xt, dev)
    if lse is None:
        lse = torch.empty((h, nq), dtype=torch.float32, device=dev)
    lp = _lse_of(lse, h, nq, dev)
    workspace, wp, wn = _room(workspace, _cross_room(dev.index, dt, nq, nk, h, hk, d, batch, 0, _in_place(qv, kv, vv)), dev)
    rc = lib.gt_cross_attn_fwd(dt, nq, nk, h, hk, d, batch, *qv, *kv, *vv, qp, kp, mp,
                               1.0 / math.sqrt(d) if scale is None else scale, *ov, lp, wp, wn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_cross_attn_fwd", rc)
    return out, lse


def gt_cross_attn_bwd(q, k, v, o, dO, lse, q_off=None, kv_off=None, key_mask=None, scale: float | None = None, dq=None,
                      dk=None, dv=None, workspace=None, stream=None):
    """Gradients of sum(o * dO) of gt_cross_attn_fwd, from its inputs and results: (dq, dk, dv), of q's type.  Rows
    outside the sequences are not written."""
    if not _is_here(q, stream):
        return _elsewhere(gt_cross_attn_bwd, q, stream,
                          (q, k, v, o, dO, lse, q_off, kv_off, key_mask, scale, dq, dk, dv, workspace))
    lib = _lib or load_library()
    nq, h, d = _three_dims("q", q)
    nk, hk, _ = _three_dims("k", k)
    xt, dev, dt = q.dtype, q.device, _type_code("q", q)
    qv, kv, vv = _heads("q", q, nq, h, d, xt, dev), _heads("k", k, nk, hk, d, xt, dev), _heads("v", v, nk, hk, d, xt, dev)
    ov, gv, lp = _heads("o", o, nq, h, d, xt, dev), _heads("dO", dO, nq, h, d, xt, dev), _lse_of(lse, h, nq, dev)
    batch, qp, kp, mp = _sequences(q_off, kv_off, nk, key_mask, dev)
    dq, dqv = _heads_result("dq", dq, nq, h, d, xt, dev)
    dk, dkv = _heads_result("dk", dk, nk, hk, d, xt, dev)
    dv, dvv = _heads_result("dv", dv, nk, hk, d, xt, dev)
    workspace, wp, wn = _room(workspace,
                              _cross_room(dev.index, dt, nq, nk, h, hk, d, batch, 1, _in_place(qv, kv, vv, gv)), dev)
    rc = lib.gt_cross_attn_bwd(dt, nq, nk, h, hk, d, batch, *qv, *kv, *vv, *ov, *gv, lp, qp, kp, mp,
                               1.0 / math.sqrt(d) if scale is None else scale, *dqv, *dkv, *dvv, wp, wn,
                               _raw_stream(dev.index))
    if rc:
        raise GtError("gt_cross_attn_bwd", rc)
    return dq, dk, dv


@functools.lru_cache(maxsize=256)
def _qk_room(device_index, d):
    return int(load_library().gt_qk_norm_workspace_size(d))


def gt_qk_norm_workspace_size(d: int) -> int:
    """Workspace bytes of gt_qk_norm_bwd (0 for a d that is not supported)."""
    return 0 if d > _MOST else int(load_library().gt_qk_norm_workspace_size(d))


def _rotation(freq, d, device):
    """(address, channels that turn) of the rotation's frequencies"""
    if freq is None:
        return None, 0
    if freq.dim() != 1 or 2 * freq.numel() > d or freq.numel() < 1:
        raise ValueError(f"freq must be fp32 [rot / 2] with 2 <= rot <= {d}, got {tuple(freq.shape)}")
    return _vector("freq", freq, freq.numel(), device), 2 * freq.numel()


def gt_qk_norm_fwd(q, k, gain_q, gain_k=None, freq=None, pos_q=None, pos_k=None, pairs: int = GT_ROT_HALVES,
                   eps: float = 1e-6, out_dtype=None, out_q=None, out_k=None, stream=None):
    """Norm of every head of q [nq][h][d] and k [nk][hk][d] (one type; k may be None): gain x / sqrt(mean x^2 + eps),
    and, with freq fp32 [rot / 2], the rotation of the first rot channels by pos * freq.  Returns (yq, yk) of out_dtype
    (default: q's type).  pos_q, pos_k int32: the rows' positions (default: their index).  pairs: channels i and
    i + rot / 2 turn together (GT_ROT_HALVES), or 2 i and 2 i + 1 (GT_ROT_PAIRS).  out_q may be q, out_k may be k."""
    if not _is_here(q, stream):
        return _elsewhere(gt_qk_norm_fwd, q, stream,
                          (q, k, gain_q, gain_k, freq, pos_q, pos_k, pairs, eps, out_dtype, out_q, out_k))
    lib = _lib or load_library()
    nq, h, d = _three_dims("q", q)
    xt, dev = q.dtype, q.device
    yt = out_dtype or (xt if out_q is None else out_q.dtype)
    fp, rot = _rotation(freq, d, dev)
    qv, gq = _heads("q", q, nq, h, d, xt, dev), _vector("gain_q", gain_q, d, dev)
    pq = None if pos_q is None else _ints("pos_q", pos_q, nq, dev)
    out_q, yqv = _heads_result("out_q", out_q, nq, h, d, yt, dev)
    keys = (1, 1, None, 0, 0, None, None, None, 0, 0)
    if k is not None:
        nk, hk, _ = _three_dims("k", k)
        kv, gk = _heads("k", k, nk, hk, d, xt, dev), _vector("gain_k", gain_k, d, dev)
        pk = None if pos_k is None else _ints("pos_k", pos_k, nk, dev)
        out_k, ykv = _heads_result("out_k", out_k, nk, hk, d, yt, dev)
        keys = (nk, hk, *kv, gk, pk, *ykv)
    elif gain_k is not None or pos_k is not None or out_k is not None:
        raise ValueError("gain_k, pos_k and out_k belong to k")
    rc = lib.gt_qk_norm_fwd(_type_code("q", q), _type_code("out_q", out_q), d, eps, fp, rot, pairs, nq, h, *qv, gq, pq, *yqv,
                            *keys, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_qk_norm_fwd", rc)
    return out_q, out_k


def gt_qk_norm_bwd(dyq, dyk, q, k, gain_q, gain_k=None, freq=None, pos_q=None, pos_k=None, pairs: int = GT_ROT_HALVES,
                   eps: float = 1e-6, dq=None, dk=None, dgain_q=None, dgain_k=None, workspace=None, stream=None):
    """Backward of gt_qk_norm_fwd from dyq and dyk (one type) and the forward's inputs: (dq, dk, dgain_q, dgain_k), dq
    and dk of q's type, the gains' gradients fp32 [d].  dyk and k may be None."""
    if not _is_here(q, stream):
        return _elsewhere(gt_qk_norm_bwd, q, stream, (dyq, dyk, q, k, gain_q, gain_k, freq, pos_q, pos_k, pairs, eps, dq, dk,
                                                      dgain_q, dgain_k, workspace))
    lib = _lib or load_library()
    nq, h, d = _three_dims("q", q)
    xt, yt, dev = q.dtype, dyq.dtype, q.device
    fp, rot = _rotation(freq, d, dev)
    qv, gq = _heads("q", q, nq, h, d, xt, dev), _vector("gain_q", gain_q, d, dev)
    dyqv = _heads("dyq", dyq, nq, h, d, yt, dev)
    pq = None if pos_q is None else _ints("pos_q", pos_q, nq, dev)
    dq, dqv = _heads_result("dq", dq, nq, h, d, xt, dev)
    dgain_q, dgq = _result("dgain_q", dgain_q, d, dev)
    keys = (1, 1, None, 0, 0, None, 0, 0, None, None, None, 0, 0, None)
    if k is not None:
        if dyk is None:
            raise ValueError("k comes with dyk")
        nk, hk, _ = _three_dims("k", k)
        kv, gk = _heads("k", k, nk, hk, d, xt, dev), _vector("gain_k", gain_k, d, dev)
        dykv = _heads("dyk", dyk, nk, hk, d, yt, dev)
        pk = None if pos_k is None else _ints("pos_k", pos_k, nk, dev)
        dk, dkv = _heads_result("dk", dk, nk, hk, d, xt, dev)
        dgain_k, dgk = _result("dgain_k", dgain_k, d, dev)
        keys = (nk, hk, *dykv, *kv, gk, pk, *dkv, dgk)
    elif any(t is not None for t in (dyk, gain_k, pos_k, dk, dgain_k)):
        raise ValueError("dyk, gain_k, pos_k, dk and dgain_k belong to k")
    workspace, wp, wn = _room(workspace, _qk_room(dev.index, d), dev)
    rc = lib.gt_qk_norm_bwd(_type_code("q", q), _type_code("dyq", dyq), d, eps, fp, rot, pairs, nq, h, *dyqv, *qv, gq, pq,
                            *dqv, dgq, *keys, wp, wn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_qk_norm_bwd", rc)
    return dq, dk, dgain_q, dgain_k


class _Grad(ctypes.Structure):
    """gt_grad of the C ABI."""
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64), ("gtype", ctypes.c_int32),
                ("otype", ctypes.c_int32)]


def _dense(t):
    """Whether t's elements fill a piece of memory, in whatever order."""
    if t.is_contiguous():
        return True
    need = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride != need:
            return False
        need *= size
    return True


class TensorList:
    """The gradients of a step, and where their clipped values go, laid out for gt_grad_clip once (gt_tensor_list).  It
    holds the memory that the tensors have now."""

    def __init__(self, grads, out=None):
        grads = [t.detach() for t in grads]
        out = grads if out is None else [t.detach() for t in out]
        if not grads or len(out) != len(grads):
            raise ValueError("gt_tensor_list needs at least one gradient, and as many outputs")
        device = grads[0].device
        table = (_Grad * len(grads))()
        for i, (g, o) in enumerate(zip(grads, out)):
            if not g.is_cuda:
                raise ValueError("libgt works on CUDA tensors only")
            if g.device != device or o.device != device:
                raise ValueError(f"gradient {i} and its output must be on {device}")
            if o.shape != g.shape or (o.stride() != g.stride() and not (g.is_contiguous() and o.is_contiguous())):
                raise ValueError(f"output {i} must have its gradient's shape and strides")
            if not _dense(g):
                raise ValueError(f"the elements of gradient {i} must fill one piece of memory")
            p, q = g.data_ptr(), o.data_ptr()
            if p == q and p and g.dtype != o.dtype:
                raise ValueError(f"output {i} is its gradient in another type")
            table[i] = _Grad(p, q, g.numel(), _type_code(f"gradient {i}", g), _type_code(f"output {i}", o))
        written = [t.data_ptr() for t in out if t.numel()]
        if len(set(written)) != len(written):
            raise ValueError("an output is listed twice")
        self.grads, self.out, self.device, self.table, self.count = grads, out, device, table, len(grads)
        self.address = ctypes.addressof(table)


def gt_tensor_list(grads, out=None) -> TensorList:
    """The handle that gt_grad_clip takes instead of lists, for programs whose gradients stay where they are."""
    return TensorList(grads, out)


@functools.lru_cache(maxsize=256)
def _clip_room(device_index, count):
    return int(load_library().gt_grad_clip_workspace_size(count))


def gt_grad_clip_workspace_size(count: int) -> int:
    """Workspace bytes of gt_grad_clip over `count` tensors."""
    return 0 if count > _MOST else int(load_library().gt_grad_clip_workspace_size(count))


def _grad_clip(tensors, max_norm, norm, workspace):
    lib = _lib or load_library()
    dev = tensors.device
    norm, np_ = _result("norm", norm, 1, dev)
    workspace, wp, wn = _room(workspace, _clip_room(dev.index, tensors.count), dev)
    rc = lib.gt_grad_clip(tensors.address, tensors.count, max_norm, np_, wp, wn, _raw_stream(dev.index))
    if rc:
        raise GtError("gt_grad_clip", rc)
    return (norm,)


def gt_grad_clip(grads, max_norm: float, out=None, norm=None, workspace=None, stream=None):
    """Norm fp32 [1] of all gradients together (a list of fp32 and bf16 tensors, or a gt_tensor_list), which are scaled
    to max_norm in place, or into `out`, where the norm exceeds it.  max_norm = inf only measures."""
    if isinstance(grads, TensorList):
        if out is not None:
            raise ValueError("a gt_tensor_list has its outputs already")
        tensors = grads
    else:
        tensors = TensorList(grads, out)
    if stream is None and tensors.device.index == _current_device():
        return _grad_clip(tensors, max_norm, norm, workspace)[0]
    if stream is not None and stream.device == tensors.device:
        for t in (*tensors.grads, *tensors.out):
            t.record_stream(stream)
    return _elsewhere(_grad_clip, tensors.grads[0], stream, (tensors, max_norm, norm, workspace))[0]


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
