"""ctypes binding of libfg8.so (the C ABI declared in include/fg8.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels.  PyTorch provides device memory and the current stream.  If the
library has not been built this module raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfg8.so")

FG8_OK, FG8_EINVAL, FG8_EUNSUPPORTED, FG8_EHIP = 0, 1, 2, 3
OUT_F32, OUT_BF16 = 0, 1
SCALE_KINDS = {"1x128": 0, "128x128": 1, "mx": 2, "1x128_t": 3}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}

_c_i64 = ctypes.c_int64
_c_i32 = ctypes.c_int32
_c_ptr = ctypes.c_void_p

_SIGNATURES = {
    "fp8_quantize": [_c_ptr, _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_ptr, _c_ptr, _c_ptr],
    "fp8_quantize_bf16": [_c_ptr, _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_ptr, _c_ptr, _c_ptr],
    "gemm_fp8_blockscaled": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int, _c_i64, _c_i64,
                             _c_i64, _c_ptr, ctypes.c_size_t, _c_ptr],
    "gemm_fp8_blockscaled_noalloc": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int,
                                     _c_i64, _c_i64, _c_i64, _c_ptr],
    "grouped_gemm_fp8_contiguous": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int,
                                    _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "grouped_gemm_fp8_contiguous_swiglu": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                           _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "grouped_gemm_fp8_kgrouped": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int,
                                  _c_i32, _c_i64, _c_i64, _c_i64, _c_ptr],
    "grouped_gemm_fp8_masked": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int,
                                _c_i32, _c_i64, _c_i64, _c_i64, _c_ptr],
    "gemm_mxfp8": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int, _c_i32, _c_i64,
                   _c_i64, _c_i64, _c_ptr],
    "grouped_gemm_mxfp8_contiguous": [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int,
                                      _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "moe_contiguous_layout_fp8": [_c_ptr, _c_i32, _c_i64, _c_i64, _c_ptr, _c_i32, _c_i32, _c_i64,
                                  _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr],
    "fg8_moe_capacity": [_c_i64, _c_i32, _c_i32],
    "grouped_gemm_bf16": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, ctypes.c_int, _c_i64,
                          _c_i64, _c_i64, _c_i32, _c_ptr],
    "grouped_gemm_bf16_dgrad": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, ctypes.c_int,
                                _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "grouped_gemm_bf16_wgrad": [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr, ctypes.c_int,
                                _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "gemm_bf16_epilogue": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, ctypes.c_int, _c_ptr, _c_i64,
                           _c_ptr, _c_ptr, _c_i64, ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_ptr,
                           ctypes.c_size_t, _c_ptr],
    "gemm_bf16_epilogue_backward": [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr, ctypes.c_int,
                                    _c_ptr, _c_ptr, ctypes.c_int, _c_ptr, _c_i64, _c_i64, _c_i64,
                                    _c_ptr, ctypes.c_size_t, _c_ptr],
    "fg8_gemm_bf16_workspace_bytes": [_c_i64, _c_i64, _c_i64],
    "fg8_gemm_bf16_backward_workspace_bytes": [_c_i64, _c_i64, _c_i64],
    "gemm_bf16_gated": [_c_ptr, _c_i64, _c_ptr, ctypes.c_int, _c_ptr, _c_ptr, _c_i64, ctypes.c_int,
                        _c_i64, _c_i64, _c_i64, _c_ptr, ctypes.c_size_t, _c_ptr],
    "grouped_gemm_bf16_gated": [_c_ptr, _c_i64, _c_ptr, _c_ptr, ctypes.c_int, _c_ptr, _c_ptr, _c_i64,
                                ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr],
    "gemm_bf16_gated_backward": [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr, ctypes.c_int, _c_ptr,
                                 _c_ptr, ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_ptr,
                                 ctypes.c_size_t, _c_ptr],
    "grouped_gemm_bf16_gated_backward": [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr,
                                         ctypes.c_int, _c_ptr, _c_ptr, ctypes.c_int, _c_i64, _c_i64,
                                         _c_i64, _c_i32, _c_ptr, ctypes.c_size_t, _c_ptr],
    "fg8_gemm_bf16_gated_workspace_bytes": [_c_i64, _c_i64, _c_i64],
    "fg8_gemm_bf16_gated_backward_workspace_bytes": [_c_i64, _c_i64, _c_i64, _c_i32],
    "int4_quantize": [_c_ptr, _c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr, _c_ptr, _c_i32, _c_ptr],
    "int4_dequantize": [_c_ptr, _c_ptr, _c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_ptr, ctypes.c_int,
                        _c_ptr],
    "gemm_bf16_int4": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, _c_i32, _c_ptr, _c_i32, ctypes.c_int,
                       _c_i32, _c_ptr, _c_i64, _c_ptr, _c_i64, ctypes.c_int, _c_i64, _c_i64, _c_i64,
                       _c_ptr],
    "grouped_gemm_bf16_int4": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, _c_i32, _c_ptr, ctypes.c_int,
                               _c_i32, _c_ptr, _c_i64, ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_i32,
                               _c_ptr],
    "linear_cross_entropy": [_c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, _c_ptr, _c_ptr, _c_i64, _c_i64,
                             _c_i64, _c_ptr, ctypes.c_size_t, _c_ptr],
    "linear_cross_entropy_backward": [_c_ptr, _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, _c_ptr, _c_ptr,
                                      _c_ptr, ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_ptr,
                                      ctypes.c_size_t, _c_ptr],
    "fg8_linear_cross_entropy_workspace_bytes": [_c_i64, _c_i64, _c_i64],
    "fg8_linear_cross_entropy_backward_workspace_bytes": [_c_i64, _c_i64, _c_i64, ctypes.c_int],
    "layer_norm": [_c_ptr, _c_i64, _c_i32, _c_ptr, _c_ptr, _c_i32, ctypes.c_float, _c_i64, _c_i64,
                   _c_ptr, _c_ptr, _c_ptr, _c_ptr],
    "layer_norm_backward": [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_i32, _c_ptr, _c_i32, _c_ptr, _c_ptr,
                            _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_size_t,
                            _c_ptr],
    "fg8_layer_norm_backward_workspace_bytes": [_c_i64, _c_i64, _c_i32],
    "moe_combine": [_c_ptr, _c_i32, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i32, _c_i64, _c_ptr,
                    _c_ptr],
    "moe_combine_backward": [_c_ptr, _c_ptr, _c_i32, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i32,
                             _c_i64, _c_ptr, _c_ptr, _c_ptr],
    "fg8_gemm_workspace_bytes": [_c_i64, _c_i64, _c_i64],
    "fg8_tile_choice": [_c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_ptr],
    "fg8_bf16_tile_choice": [_c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_ptr],
    "fg8_bf16_fused_tile_choice": [_c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_ptr],
    "fg8_last_error": [],
    "fg8_version": [],
}
_RESTYPES = {"fg8_gemm_workspace_bytes": ctypes.c_size_t, "fg8_last_error": ctypes.c_char_p,
             "fg8_moe_capacity": ctypes.c_int64,
             "fg8_gemm_bf16_workspace_bytes": ctypes.c_size_t,
             "fg8_gemm_bf16_backward_workspace_bytes": ctypes.c_size_t,
             "fg8_gemm_bf16_gated_workspace_bytes": ctypes.c_size_t,
             "fg8_gemm_bf16_gated_backward_workspace_bytes": ctypes.c_size_t,
             "fg8_linear_cross_entropy_workspace_bytes": ctypes.c_size_t,
             "fg8_linear_cross_entropy_backward_workspace_bytes": ctypes.c_size_t,
             "fg8_layer_norm_backward_workspace_bytes": ctypes.c_size_t}

_lib = None
_lock = threading.Lock()


class Fg8Error(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"fg8 status {status}: {message}")
        self.status = status


def lib():
    """Load libfg8.so once.  Raises if it is missing: the HIP path has no
    substitute."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is not built; run "
                                       "`python -m moe_grouped_gemm_fp8_amd.build`")
                L = ctypes.CDLL(LIB_PATH)
                for name, args in _SIGNATURES.items():
                    fn = getattr(L, name)
                    fn.argtypes = args
                    fn.restype = _RESTYPES.get(name, ctypes.c_int)
                _lib = L
    return _lib


def _check(status):
    if status != FG8_OK:
        raise Fg8Error(status, lib().fg8_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _here(t, name):
    """The library launches on the current device and goes by its size: every
    operand has to lie there."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is "
                         f"cuda:{torch._C._cuda_getDevice()}")


def _dev(t, dtype, name):
    _here(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _fp8(t, name):
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return _dev(t, torch.uint8, name)


def _out_code(dtype):
    if dtype == torch.float32:
        return OUT_F32
    if dtype == torch.bfloat16:
        return OUT_BF16
    raise TypeError("output dtype must be float32 or bfloat16")


def version() -> int:
    return lib().fg8_version()


def tile_choice(mode, m, n, k, groups=1, num_cus=None):
    """The tiling the library picks for a GEMM of this shape (fg8_tile_choice;
    mode 0 dense, 1 contiguous, 2 masked, 3 K-grouped): dict of bm, bn,
    splits, grid, raster.  num_cus defaults to the current device's."""
    if num_cus is None:
        num_cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = (ctypes.c_int32 * 5)()
    _check(lib().fg8_tile_choice(mode, m, n, k, groups, num_cus, ctypes.cast(out, ctypes.c_void_p)))
    return dict(zip(("bm", "bn", "splits", "grid", "raster"), list(out)))


BF16_PRODUCTS = ("gemm_bf16_epilogue", "dx", "dw", "grouped_gemm_bf16", "grouped_gemm_bf16_dgrad", "grouped_gemm_bf16_wgrad")


BF16_FUSED_PRODUCTS = ("gemm_bf16_gated", "grouped_gemm_bf16_gated", "linear_cross_entropy", "linear_cross_entropy_backward",
                       "linear_cross_entropy_dx")


def bf16_tile_choice(product, m, n, k, groups=1, num_cus=None):
    """The tiling the library picks for a BF16 product (fg8_bf16_tile_choice,
    fg8_bf16_fused_tile_choice): one of BF16_PRODUCTS ("dx" and "dw" of
    gemm_bf16_epilogue_backward) or of BF16_FUSED_PRODUCTS (the loss's backward
    pass's logits and its dx, n the vocabulary) with m rows, n, k and experts as
    that call takes them; dict of bm, bn, splits, persistent.  num_cus defaults to
    the current device's."""
    if num_cus is None:
        num_cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = (ctypes.c_int32 * 4)()
    fused = product in BF16_FUSED_PRODUCTS
    choose = lib().fg8_bf16_fused_tile_choice if fused else lib().fg8_bf16_tile_choice
    _check(choose((BF16_FUSED_PRODUCTS if fused else BF16_PRODUCTS).index(product), m, n, k, groups, num_cus,
                  ctypes.cast(out, ctypes.c_void_p)))
    return dict(zip(("bm", "bn", "splits", "persistent"), list(out)))


# --------------------------------------------------------------- quantize
def fp8_quantize(x, kind="1x128", q=None, scales=None):
    """x float32 or bfloat16 [..., rows, cols] -> (q uint8, scales); see fg8.h
    for layouts ("1x128_t": groups of 128 rows, q [..., cols, rows]).  A
    bfloat16 source quantizes exactly like its float32 value."""
    bf16 = x.dtype == torch.bfloat16
    _dev(x, torch.bfloat16 if bf16 else torch.float32, "x")
    code = SCALE_KINDS[kind]
    *lead, rows, cols = x.shape
    batch = 1
    for d in lead:
        batch *= d
    if q is None:
        shape = (*lead, cols, rows) if kind == "1x128_t" else x.shape
        q = torch.empty(shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        if kind == "1x128_t":
            scales = torch.empty((*lead, rows // 128, cols), dtype=torch.float32, device=x.device)
        elif kind == "1x128":
            scales = torch.empty((*lead, cols // 128, rows), dtype=torch.float32, device=x.device)
        elif kind == "128x128":
            scales = torch.empty((*lead, -(-rows // 128), cols // 128), dtype=torch.float32,
                                 device=x.device)
        else:
            scales = torch.empty((*lead, rows, cols // 32), dtype=torch.uint8, device=x.device)
    fn = lib().fp8_quantize_bf16 if bf16 else lib().fp8_quantize
    _check(fn(_ptr(x), batch, rows, cols, code, _ptr(q), _ptr(scales), _stream()))
    return q, scales


# --------------------------------------------------------------- GEMMs
def gemm_workspace_bytes(m, n, k) -> int:
    return int(lib().fg8_gemm_workspace_bytes(m, n, k))


#: The arrival counters at a workspace's front (kSplitKCounterBytes of the
#: kernels): all of it that has to be zero before its first use.
WS_COUNTER_BYTES = 4096
#: The largest workspace that is kept.  Counters and partial tiles of a split
#: product take 34 MB at most (two 128 x 128 FP32 tiles a CU); what goes beyond
#: is a backward pass's dz, which grows with the call and is its alone.
WS_KEEP_BYTES = 64 << 20

_ws_cache = {}


def _stream_of(t):
    """The current stream of t's device, as a number."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _new_workspace(nbytes, t):
    ws = t.new_empty(nbytes, dtype=torch.uint8)
    ws[:WS_COUNTER_BYTES].zero_()
    return ws


def _workspace_of(nbytes, t, stream):
    """A workspace per (t's device, stream, calling thread) with its counters at
    zero, as (tensor, pointer, bytes); the kernels leave them so, and it is reused
    as is.  (Threads that share a stream may enqueue their calls' kernels in turn,
    and a call of several keeps data here between them.)  One above WS_KEEP_BYTES
    goes back with the call.  A call recorded in a graph gets one of its own, with
    its arrival counters cleared by the graph, and leaves nothing here: a cached one
    may be replaced while the graph lives, and one that a graph allocated belongs to
    the graph, whose clearing has only been recorded."""
    if nbytes == 0:
        return None, None, 0
    if nbytes > WS_KEEP_BYTES or torch.cuda.is_current_stream_capturing():
        ws = _new_workspace(nbytes, t)
    else:
        key = (t.device, stream, threading.get_ident())
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            if ws is None:               # (what threads kept that have ended)
                alive = {th.ident for th in threading.enumerate()}
                for other in list(_ws_cache):
                    if other[2] not in alive and other[2] != key[2]:
                        _ws_cache.pop(other, None)
            ws = None
            _ws_cache.pop(key, None)     # (its memory serves the larger one)
            ws = _ws_cache[key] = _new_workspace(nbytes, t)
    return ws, ws.data_ptr(), ws.numel()


def _workspace_given(ws):
    """A caller's workspace as (pointer, bytes)."""
    _dev(ws, ws.dtype, "workspace")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def gemm_fp8_blockscaled(a, sa, b, sb, out_dtype=torch.bfloat16, out=None, workspace=None):
    """D [m, n] = A B^T with a [m, k] e4m3, sa [k/128, m], b [n, k], sb [ceil(n/128), k/128].
    Recorded in a graph without a workspace, a split product clears the counters
    of one of its own on every replay; a zero-filled `workspace` (see
    gemm_workspace_bytes) that the caller keeps for the graph saves that."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or sa.shape != (k // 128, m) or sb.shape != (-(-n // 128), k // 128):
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    stream = _stream_of(a)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(gemm_workspace_bytes(m, n, k), a, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(lib().gemm_fp8_blockscaled(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out),
                                      _out_code(out.dtype), m, n, k, ws, ws_bytes, stream))
    return out


def gemm_fp8_blockscaled_noalloc(a, sa, b, sb, out_dtype=torch.bfloat16, out=None):
    """gemm_fp8_blockscaled without a workspace: the split-K scratch is the
    library's static per-GPU array (see fg8.h).  `out` must be given by
    callers that cannot allocate; calls that overlap on one GPU race."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or sa.shape != (k // 128, m) or sb.shape != (-(-n // 128), k // 128):
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    if out.shape != (m, n):
        raise ValueError("output shape disagrees")
    _check(lib().gemm_fp8_blockscaled_noalloc(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out),
                                              _out_code(out.dtype), m, n, k, _stream()))
    return out


def grouped_gemm_fp8_contiguous(a, sa, b, sb, block_expert, out_dtype=torch.bfloat16, out=None):
    """Contiguous layout: a [m_total, k], sa [k/128, m_total], b [E, n, k],
    sb [E, ceil(n/128), k/128], block_expert int32 [m_total/128]."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    _dev(block_expert, torch.int32, "block_expert")
    m, k = a.shape
    E, n, kb = b.shape
    if kb != k or sa.shape != (k // 128, m) or sb.shape != (E, -(-n // 128), k // 128) \
            or block_expert.shape != (m // 128,):
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    _check(lib().grouped_gemm_fp8_contiguous(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                                             _ptr(block_expert), _ptr(out), _out_code(out.dtype),
                                             m, n, k, E, _stream()))
    return out


def grouped_gemm_fp8_contiguous_swiglu(a, sa, b, sb, block_expert, q_out=None, s_out=None):
    """The contiguous grouped GEMM with W1 (rows interleaved in 128-row gate /
    up blocks, see fg8.h) and the SiLU-gated activation plus its 1x128
    quantization fused into the epilogue: a [m_total, k], sa [k/128, m_total],
    b [E, n, k], sb [E, n/128, k/128], block_expert int32 [m_total/128] ->
    (q_out uint8 [m_total, n/2], s_out float32 [n/256, m_total]).  Rows of
    skipped blocks (expert id out of range) are left as they were."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    _dev(block_expert, torch.int32, "block_expert")
    m, k = a.shape
    E, n, kb = b.shape
    if kb != k or sa.shape != (k // 128, m) or sb.shape != (E, -(-n // 128), k // 128) \
            or block_expert.shape != (m // 128,):
        raise ValueError("operand shapes disagree")
    if q_out is None:
        q_out = torch.empty((m, n // 2), dtype=torch.uint8, device=a.device)
    if s_out is None:
        s_out = torch.empty((n // 256, m), dtype=torch.float32, device=a.device)
    _dev(q_out, torch.uint8, "q_out"); _dev(s_out, torch.float32, "s_out")
    if q_out.shape != (m, n // 2) or s_out.shape != (n // 256, m):
        raise ValueError("output shapes disagree")
    _check(lib().grouped_gemm_fp8_contiguous_swiglu(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                                                    _ptr(block_expert), _ptr(q_out), _ptr(s_out),
                                                    m, n, k, E, _stream()))
    return q_out, s_out


def grouped_gemm_fp8_kgrouped(a, sa, b, sb, k_offsets, out_dtype=torch.float32, out=None):
    """Weight-gradient layout: a [m, k_total], sa [k_total/128, m], b [n, k_total],
    sb [k_total/128, n] (1x128 along K on both), k_offsets int32 [G + 1]
    (device) -> d [G, m, n] with d[g] = A[:, K_g] B[:, K_g]^T."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    _dev(k_offsets, torch.int32, "k_offsets")
    m, k = a.shape
    n = b.shape[0]
    G = k_offsets.shape[0] - 1
    if b.shape != (n, k) or sa.shape != (k // 128, m) or sb.shape != (k // 128, n) or G < 1:
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.empty((G, m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    if out.shape != (G, m, n):
        raise ValueError("output shape disagrees")
    _check(lib().grouped_gemm_fp8_kgrouped(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(k_offsets),
                                           _ptr(out), _out_code(out.dtype), G, m, n, k, _stream()))
    return out


def grouped_gemm_fp8_masked(a, sa, b, sb, valid_rows, out_dtype=torch.bfloat16, out=None):
    """Masked layout: a [E, cap, k], sa [E, k/128, cap], b [E, n, k],
    sb [E, ceil(n/128), k/128], valid_rows int32 [E] (device).  Rows at or
    past valid_rows[e] of `out` are left as they were."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.float32, "sa"); _dev(sb, torch.float32, "sb")
    _dev(valid_rows, torch.int32, "valid_rows")
    E, cap, k = a.shape
    n = b.shape[1]
    if b.shape != (E, n, k) or sa.shape != (E, k // 128, cap) \
            or sb.shape != (E, -(-n // 128), k // 128) or valid_rows.shape != (E,):
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.zeros((E, cap, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    _check(lib().grouped_gemm_fp8_masked(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(valid_rows),
                                         _ptr(out), _out_code(out.dtype), E, cap, n, k, _stream()))
    return out


def gemm_mxfp8(a, sa, b, sb, valid_rows=None, out_dtype=torch.bfloat16, out=None):
    """MXFP8: a [G, m, k], sa uint8 [G, m, k/32], b [G, n, k], sb uint8 [G, n, k/32],
    valid_rows None or int32 [G] (device)."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.uint8, "sa"); _dev(sb, torch.uint8, "sb")
    G, m, k = a.shape
    n = b.shape[1]
    if b.shape != (G, n, k) or sa.shape != (G, m, k // 32) or sb.shape != (G, n, k // 32):
        raise ValueError("operand shapes disagree")
    if valid_rows is not None:
        _dev(valid_rows, torch.int32, "valid_rows")
    if out is None:
        alloc = torch.empty if valid_rows is None else torch.zeros
        out = alloc((G, m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    _check(lib().gemm_mxfp8(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(valid_rows), _ptr(out),
                            _out_code(out.dtype), G, m, n, k, _stream()))
    return out


def grouped_gemm_mxfp8_contiguous(a, sa, b, sb, block_expert, out_dtype=torch.bfloat16, out=None):
    """Contiguous layout with MXFP8 operands: a [m_total, k], sa uint8
    [m_total, k/32], b [E, n, k], sb uint8 [E, n, k/32], block_expert int32
    [m_total/128]."""
    _fp8(a, "a"); _fp8(b, "b")
    _dev(sa, torch.uint8, "sa"); _dev(sb, torch.uint8, "sb")
    _dev(block_expert, torch.int32, "block_expert")
    m, k = a.shape
    E, n, kb = b.shape
    if kb != k or sa.shape != (m, k // 32) or sb.shape != (E, n, k // 32) \
            or block_expert.shape != (m // 128,):
        raise ValueError("operand shapes disagree")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _dev(out, out.dtype, "out")
    _check(lib().grouped_gemm_mxfp8_contiguous(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                                               _ptr(block_expert), _ptr(out),
                                               _out_code(out.dtype), m, n, k, E, _stream()))
    return out


# --------------------------------------------------------------- MoE routing
def moe_capacity(tokens, topk, num_experts) -> int:
    """Rows of a contiguous layout that hold any routing of these sizes."""
    return int(lib().fg8_moe_capacity(tokens, topk, num_experts))


def moe_contiguous_layout_fp8(x, topk_ids, num_experts, m_cap=None, out=None):
    """x float32 or bfloat16 [tokens, hidden], topk_ids int32 [tokens, topk]
    (device) -> dict of q uint8 [m_cap, hidden], sa [hidden/128, m_cap],
    block_expert int32 [m_cap/128], row_token int32 [m_cap], token_row int32
    [tokens, topk], expert_offsets int32 [E + 1], expert_counts int32 [E], all
    on the device: the operands of grouped_gemm_fp8_contiguous plus the row
    map and its inverse.  `out`, a
    dict like the one returned, gives the buffers to fill."""
    bf16 = x.dtype == torch.bfloat16
    _dev(x, torch.bfloat16 if bf16 else torch.float32, "x")
    _dev(topk_ids, torch.int32, "topk_ids")
    tokens, hidden = x.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != tokens:
        raise ValueError("topk_ids must be [tokens, topk]")
    topk = topk_ids.shape[1]
    if m_cap is None:
        m_cap = moe_capacity(tokens, topk, num_experts)
    dev = x.device
    shapes = {"q": ((m_cap, hidden), torch.uint8), "sa": ((hidden // 128, m_cap), torch.float32),
              "block_expert": ((m_cap // 128,), torch.int32), "row_token": ((m_cap,), torch.int32),
              "token_row": ((tokens, topk), torch.int32),
              "expert_offsets": ((num_experts + 1,), torch.int32),
              "expert_counts": ((num_experts,), torch.int32)}
    if out is not None:
        for name, (shape, dtype) in shapes.items():
            _dev(out[name], dtype, name)
            if tuple(out[name].shape) != shape:
                raise ValueError(f"{name} must have shape {shape}")
    else:
        out = {name: torch.empty(shape, dtype=dtype, device=dev)
               for name, (shape, dtype) in shapes.items()}
    _check(lib().moe_contiguous_layout_fp8(
        _ptr(x), int(bf16), tokens, hidden, _ptr(topk_ids), topk, num_experts, m_cap,
        _ptr(out["q"]), _ptr(out["sa"]), _ptr(out["block_expert"]), _ptr(out["row_token"]),
        _ptr(out["token_row"]), _ptr(out["expert_offsets"]), _ptr(out["expert_counts"]),
        _stream()))
    return out


# ------------------------------------------- BF16 products over ragged runs
# These calls are made many times a layer and some run for a few microseconds,
# so their host side is kept short: the stream as a plain number, outputs from
# an operand's new_empty.
def _rows(t, dtype, name):
    """Row stride of a 2-D tensor whose rows are contiguous but may be part of
    wider ones."""
    _here(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, cols = t.shape
    if rows <= 1:   # (a single row's stride means nothing)
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        return -(-cols // 8) * 8
    ld = t.stride(0)
    if ld < cols or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}'s rows must be contiguous and apart")
    return ld


def _out_rows(out, shape, dtype, like, name="out"):
    """(tensor, row stride, dtype code) of a given or new 2-D output."""
    if out is None:
        return like.new_empty(shape, dtype=dtype), shape[1], _out_code(dtype)
    code = _out_code(out.dtype)
    ld = _rows(out, out.dtype, name)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return out, (ld if out.shape[0] > 1 else shape[1]), code


def _experts(w, row_offsets):
    _dev(w, torch.bfloat16, "w")
    _dev(row_offsets, torch.int32, "row_offsets")
    if w.dim() != 3 or row_offsets.shape != (w.shape[0] + 1,):
        raise ValueError("w must be [E, n, k] and row_offsets [E + 1]")
    return w.shape


def grouped_gemm_bf16(x, w, row_offsets, out_dtype=torch.bfloat16, out=None):
    """Expert products over ragged row runs: x bf16 [rows, k] (rows may be
    strided), w bf16 [E, n, k], row_offsets int32 [E + 1] (device), rows
    row_offsets[e] .. row_offsets[e + 1] - 1 belonging to expert e -> y
    [rows, n] with y[r] = x[r] w[e]^T; rows of no run are zeros."""
    E, n, k = _experts(w, row_offsets)
    ldx = _rows(x, torch.bfloat16, "x")
    rows = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("operand shapes disagree")
    out, ldy, code = _out_rows(out, (rows, n), out_dtype, x)
    _check(lib().grouped_gemm_bf16(x.data_ptr(), ldx, w.data_ptr(), row_offsets.data_ptr(),
                                   out.data_ptr(), ldy, code, rows, n, k, E, _stream_of(x)))
    return out


def grouped_gemm_bf16_dgrad(dy, w, row_offsets, out_dtype=torch.bfloat16, out=None):
    """Input gradient of grouped_gemm_bf16: dy bf16 [rows, n], w bf16 [E, n, k]
    -> dx [rows, k] with dx[r] = dy[r] w[e]; rows of no run are zeros."""
    E, n, k = _experts(w, row_offsets)
    lddy = _rows(dy, torch.bfloat16, "dy")
    rows = dy.shape[0]
    if dy.shape[1] != n:
        raise ValueError("operand shapes disagree")
    out, ldx, code = _out_rows(out, (rows, k), out_dtype, dy)
    _check(lib().grouped_gemm_bf16_dgrad(dy.data_ptr(), lddy, w.data_ptr(), row_offsets.data_ptr(),
                                         out.data_ptr(), ldx, code, rows, n, k, E, _stream_of(dy)))
    return out


def grouped_gemm_bf16_wgrad(dy, x, row_offsets, out_dtype=torch.float32, out=None):
    """Weight gradient of grouped_gemm_bf16: dy bf16 [rows, n], x bf16
    [rows, k], row_offsets int32 [E + 1] (device) -> dw [E, n, k] with dw[e] =
    the sum of dy[r]^T x[r] over expert e's rows (zeros for an empty run)."""
    _dev(row_offsets, torch.int32, "row_offsets")
    lddy, ldx = _rows(dy, torch.bfloat16, "dy"), _rows(x, torch.bfloat16, "x")
    rows, n = dy.shape
    k = x.shape[1]
    E = row_offsets.numel() - 1
    if x.shape[0] != rows or row_offsets.dim() != 1 or E < 1:
        raise ValueError("operand shapes disagree")
    if out is None:
        out = dy.new_empty((E, n, k), dtype=out_dtype)
    _dev(out, out.dtype, "out")
    if out.shape != (E, n, k):
        raise ValueError("output shape disagrees")
    _check(lib().grouped_gemm_bf16_wgrad(dy.data_ptr(), lddy, x.data_ptr(), ldx,
                                         row_offsets.data_ptr(), out.data_ptr(),
                                         _out_code(out.dtype), rows, n, k, E, _stream_of(dy)))
    return out


# ------------------------------------------- BF16 product with an epilogue
def _param(t, cols, name):
    """(pointer, is bf16) of an optional FP32 or BF16 vector."""
    if t is None:
        return None, 0
    bf16 = t.dtype == torch.bfloat16
    _dev(t, torch.bfloat16 if bf16 else torch.float32, name)
    if t.shape != (cols,):
        raise ValueError(f"{name} must have shape ({cols},)")
    return t.data_ptr(), int(bf16)


def gemm_bf16_epilogue(x, w, bias=None, residual=None, activation="none", save_z=False,
                       out_dtype=torch.bfloat16, out=None, workspace=None):
    """y = act(x w^T + bias) + residual in one kernel: x bf16 [m, k], w bf16
    [n, k], bias float32 or bfloat16 [n], residual bf16 [m, n], activation
    "none", "relu", "silu" or "gelu" (the erf form).  Returns y, or (y, z) with
    save_z, z = x w^T + bias in bf16 for the backward pass.  x, residual and
    out may have strided rows; out may be the residual."""
    act = ACTIVATIONS[activation]
    _dev(w, torch.bfloat16, "w")
    ldx = _rows(x, torch.bfloat16, "x")
    m, k = x.shape
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError("operand shapes disagree")
    n = w.shape[0]
    bias_ptr, bias_bf16 = _param(bias, n, "bias")
    res_ptr, ldr = None, n
    if residual is not None:
        ldr = _rows(residual, torch.bfloat16, "residual")
        if residual.shape != (m, n):
            raise ValueError("residual must have the output's shape")
        res_ptr = residual.data_ptr()
        if m == 1:
            ldr = n
    out, ldy, code = _out_rows(out, (m, n), out_dtype, x)
    z = x.new_empty((m, n)) if save_z else None
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(L.fg8_gemm_bf16_workspace_bytes(m, n, k), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.gemm_bf16_epilogue(x.data_ptr(), ldx, w.data_ptr(), bias_ptr, bias_bf16, act, res_ptr,
                                ldr, z.data_ptr() if save_z else None, out.data_ptr(), ldy, code, m,
                                n, k, ws, ws_bytes, stream))
    return (out, z) if save_z else out


def gemm_bf16_epilogue_backward(dy, x, w, z=None, activation="none", dw_dtype=torch.bfloat16,
                                needs=(True, True, True), workspace=None):
    """Gradients of act(x w^T + bias) (the residual's is dy itself): dy bf16
    [m, n], x bf16 [m, k], w bf16 [n, k], z bf16 [m, n] as saved -> (dx bf16
    [m, k], dw dw_dtype [n, k], dbias float32 [n]); `needs` leaves out (None)
    what is not wanted.  Behind "silu" and "gelu" dx and a bfloat16 dw take dz
    rounded to bfloat16, a float32 dw to 2^-16 (a second product)."""
    act = ACTIVATIONS[activation]
    _dev(w, torch.bfloat16, "w")
    lddy, ldx = _rows(dy, torch.bfloat16, "dy"), _rows(x, torch.bfloat16, "x")
    m, k = x.shape
    n = w.shape[0]
    if w.shape != (n, k) or dy.shape != (m, n):
        raise ValueError("operand shapes disagree")
    if act:
        if z is None:
            raise ValueError("z is needed for the activation's slope")
        _dev(z, torch.bfloat16, "z")
        if z.shape != (m, n):
            raise ValueError("z must have dy's shape")
    dx = x.new_empty((m, k)) if needs[0] else None
    dw = x.new_empty((n, k), dtype=dw_dtype) if needs[1] else None
    db = x.new_empty(n, dtype=torch.float32) if needs[2] else None
    if m == 0:     # sums over no rows
        return dx, dw if dw is None else dw.zero_(), db if db is None else db.zero_()
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(L.fg8_gemm_bf16_backward_workspace_bytes(m, n, k), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.gemm_bf16_epilogue_backward(
        dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), _ptr(z), act, _ptr(dx), _ptr(dw),
        _out_code(dw_dtype), _ptr(db), m, n, k, ws, ws_bytes, stream))
    return dx, dw, db


# --------------------------------------------- gated feed-forward products
def _gated_weights(w, k, lead):
    _dev(w, torch.bfloat16, "w")
    if w.dim() != 2 + lead or w.shape[-1] != k or w.shape[-2] % 2 or w.shape[-2] == 0:
        raise ValueError("w must be " + ("[E, 2 n, k]" if lead else "[2 n, k]") + " with x's k")
    return w.shape[-2] // 2


def _run_offsets(w, row_offsets):
    _dev(row_offsets, torch.int32, "row_offsets")
    if row_offsets.shape != (w.shape[0] + 1,):
        raise ValueError("row_offsets must be [E + 1]")
    return w.shape[0]


def gemm_bf16_gated(x, w, activation="silu", save_z=False, out_dtype=torch.bfloat16, out=None,
                    workspace=None):
    """h = act(x wg^T) * (x wu^T) in one kernel: x bf16 [m, k] (rows may be
    strided), w bf16 [2 n, k] with wg the first n rows and wu the others,
    activation as gemm_bf16_epilogue's.  Returns h [m, n], or (h, z) with
    save_z, z = x w^T in bf16 [m, 2 n] for the backward pass."""
    act = ACTIVATIONS[activation]
    ldx = _rows(x, torch.bfloat16, "x")
    m, k = x.shape
    n = _gated_weights(w, k, 0)
    out, ldh, code = _out_rows(out, (m, n), out_dtype, x)
    z = x.new_empty((m, 2 * n)) if save_z else None
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(L.fg8_gemm_bf16_gated_workspace_bytes(m, n, k), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.gemm_bf16_gated(x.data_ptr(), ldx, w.data_ptr(), act, z.data_ptr() if save_z else None,
                             out.data_ptr(), ldh, code, m, n, k, ws, ws_bytes, stream))
    return (out, z) if save_z else out


def grouped_gemm_bf16_gated(x, w, row_offsets, activation="silu", save_z=False,
                            out_dtype=torch.bfloat16, out=None):
    """gemm_bf16_gated over ragged row runs, as grouped_gemm_bf16: w bf16
    [E, 2 n, k], row_offsets int32 [E + 1] (device); rows of no run are zeros
    (of z too)."""
    act = ACTIVATIONS[activation]
    ldx = _rows(x, torch.bfloat16, "x")
    rows, k = x.shape
    n = _gated_weights(w, k, 1)
    E = _run_offsets(w, row_offsets)
    out, ldh, code = _out_rows(out, (rows, n), out_dtype, x)
    z = x.new_empty((rows, 2 * n)) if save_z else None
    _check(lib().grouped_gemm_bf16_gated(x.data_ptr(), ldx, w.data_ptr(), row_offsets.data_ptr(), act,
                                         z.data_ptr() if save_z else None, out.data_ptr(), ldh, code,
                                         rows, n, k, E, _stream_of(x)))
    return (out, z) if save_z else out


def _gated_backward_args(dh, x, w, z, n):
    lddh, ldx = _rows(dh, torch.bfloat16, "dh"), _rows(x, torch.bfloat16, "x")
    _dev(z, torch.bfloat16, "z")
    if dh.shape != (x.shape[0], n) or z.shape != (x.shape[0], 2 * n):
        raise ValueError("dh must be [m, n] and z [m, 2 n]")
    return lddh, ldx


def gemm_bf16_gated_backward(dh, x, w, z, activation="silu", dw_dtype=torch.bfloat16,
                             needs=(True, True), workspace=None):
    """Gradients of gemm_bf16_gated: dh bf16 [m, n], x, w and z as the forward
    pass had and saved them -> (dx bf16 [m, k], dw dw_dtype [2 n, k]); `needs`
    leaves out (None) what is not wanted.  dx and a bfloat16 dw take dz rounded
    to bfloat16, a float32 dw to 2^-16 (a second product)."""
    act = ACTIVATIONS[activation]
    m, k = x.shape
    n = _gated_weights(w, k, 0)
    lddh, ldx = _gated_backward_args(dh, x, w, z, n)
    dx = x.new_empty((m, k)) if needs[0] else None
    dw = w.new_empty(w.shape, dtype=dw_dtype) if needs[1] else None
    if m == 0:     # sums over no rows
        return dx, dw if dw is None else dw.zero_()
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(
            L.fg8_gemm_bf16_gated_backward_workspace_bytes(m, n, k, 0), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.gemm_bf16_gated_backward(dh.data_ptr(), lddh, x.data_ptr(), ldx, w.data_ptr(), z.data_ptr(),
                                      act, _ptr(dx), _ptr(dw), _out_code(dw_dtype), m, n, k, ws, ws_bytes,
                                      stream))
    return dx, dw


def grouped_gemm_bf16_gated_backward(dh, x, w, z, row_offsets, activation="silu",
                                     dw_dtype=torch.float32, needs=(True, True), workspace=None):
    """Gradients of grouped_gemm_bf16_gated: dh bf16 [rows, n], z bf16
    [rows, 2 n] as saved -> (dx bf16 [rows, k], zeros in rows of no run, dw
    dw_dtype [E, 2 n, k], zeros for an empty run).  The rest as
    gemm_bf16_gated_backward."""
    act = ACTIVATIONS[activation]
    rows, k = x.shape
    n = _gated_weights(w, k, 1)
    E = _run_offsets(w, row_offsets)
    lddh, ldx = _gated_backward_args(dh, x, w, z, n)
    dx = x.new_empty((rows, k)) if needs[0] else None
    dw = w.new_empty(w.shape, dtype=dw_dtype) if needs[1] else None
    if rows == 0:
        return dx, dw if dw is None else dw.zero_()
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(
            L.fg8_gemm_bf16_gated_backward_workspace_bytes(rows, n, k, E), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.grouped_gemm_bf16_gated_backward(
        dh.data_ptr(), lddh, x.data_ptr(), ldx, w.data_ptr(), z.data_ptr(), row_offsets.data_ptr(), act,
        _ptr(dx), _ptr(dw), _out_code(dw_dtype), rows, n, k, E, ws, ws_bytes, stream))
    return dx, dw


# ------------------------------------------------------- weights in 4 bits
def int4_quantize(w, group=128, scale_dtype=torch.float32):
    """w float32 or bfloat16 [..., n, k] -> (q uint8 [..., n, k / 2], scales
    scale_dtype (float32 or bfloat16) [..., k / group, n]): 4-bit codes, each
    group of 32, 64 or 128 columns with a scale of amax / 7; see fg8.h."""
    bf16 = w.dtype == torch.bfloat16
    _dev(w, torch.bfloat16 if bf16 else torch.float32, "w")
    if w.dim() < 2 or group < 1:
        raise ValueError("w must be [..., n, k], group 32, 64 or 128")
    *lead, n, k = w.shape
    code = _out_code(scale_dtype)
    q = w.new_empty((*lead, n, k // 2), dtype=torch.uint8)
    scales = w.new_empty((*lead, k // group, n), dtype=scale_dtype)
    _check(lib().int4_quantize(w.data_ptr(), int(bf16), math.prod(lead), n, k, group, q.data_ptr(),
                               scales.data_ptr(), code, _stream_of(w)))
    return q, scales


def _int4(q, scales, lead):
    """(n, k, group, scales are bf16) of codes [..., n, k / 2] and their scales."""
    _dev(q, torch.uint8, "q")
    bf16 = scales.dtype == torch.bfloat16
    _dev(scales, torch.bfloat16 if bf16 else torch.float32, "scales")
    if q.dim() < 2 or (lead is not None and q.dim() != 2 + lead):
        raise ValueError("q must be " + ("[..., n, k / 2]" if lead is None else "[E, n, k / 2]" if lead else "[n, k / 2]"))
    n, k = q.shape[-2], 2 * q.shape[-1]
    if scales.dim() != q.dim() or scales.shape[:-2] != q.shape[:-2] or scales.shape[-1] != n or scales.shape[-2] == 0 \
            or k % scales.shape[-2]:
        raise ValueError("scales must be [..., k / group, n] for q [..., n, k / 2]")
    return n, k, k // scales.shape[-2], int(bf16)


def int4_dequantize(q, scales, out_dtype=torch.bfloat16):
    """The values [..., n, k] that codes and scales stand for, as int4_quantize
    returned them (for the BF16 products of many rows)."""
    n, k, group, bf16 = _int4(q, scales, None)
    w = q.new_empty((*q.shape[:-1], k), dtype=out_dtype)
    _check(lib().int4_dequantize(q.data_ptr(), scales.data_ptr(), bf16, math.prod(q.shape[:-2]), n, k,
                                 group, w.data_ptr(), _out_code(out_dtype), _stream_of(q)))
    return w


def gemm_bf16_int4(x, q, scales, bias=None, residual=None, activation="none", gated=False,
                   out_dtype=torch.bfloat16, out=None):
    """y = act(x W^T + bias) + residual for few rows, W [n, k] in 4 bits as
    int4_quantize returns it: x bf16 [m, k], the rest as gemm_bf16_epilogue.
    gated: W [2 n, k], y = act(x Wg^T) * (x Wu^T) as gemm_bf16_gated, without bias
    and residual."""
    act = ACTIVATIONS[activation]
    wide, k, group, s_bf16 = _int4(q, scales, 0)
    ldx = _rows(x, torch.bfloat16, "x")
    m = x.shape[0]
    if x.shape[1] != k or (gated and wide % 2):
        raise ValueError("operand shapes disagree")
    n = wide // 2 if gated else wide
    if gated and (bias is not None or residual is not None):
        raise ValueError("a gated product takes neither bias nor residual")
    bias_ptr, bias_bf16 = _param(bias, n, "bias")
    res_ptr, ldr = None, n
    if residual is not None:
        ldr = _rows(residual, torch.bfloat16, "residual")
        if residual.shape != (m, n):
            raise ValueError("residual must have the output's shape")
        res_ptr = residual.data_ptr()
        if m == 1:
            ldr = n
    out, ldy, code = _out_rows(out, (m, n), out_dtype, x)
    _check(lib().gemm_bf16_int4(x.data_ptr(), ldx, q.data_ptr(), scales.data_ptr(), s_bf16, group, bias_ptr,
                                bias_bf16, act, int(gated), res_ptr, ldr, out.data_ptr(), ldy, code, m, n, k,
                                _stream_of(x)))
    return out


def grouped_gemm_bf16_int4(x, q, scales, row_offsets, activation="none", gated=False,
                           out_dtype=torch.bfloat16, out=None):
    """gemm_bf16_int4 over ragged row runs, as grouped_gemm_bf16: q [E, n, k / 2]
    (gated: 2 n), scales [E, k / group, n], row_offsets int32 [E + 1] (device);
    rows of no run are zeros."""
    act = ACTIVATIONS[activation]
    wide, k, group, s_bf16 = _int4(q, scales, 1)
    ldx = _rows(x, torch.bfloat16, "x")
    rows = x.shape[0]
    if x.shape[1] != k or (gated and wide % 2):
        raise ValueError("operand shapes disagree")
    n = wide // 2 if gated else wide
    E = _run_offsets(q, row_offsets)
    out, ldy, code = _out_rows(out, (rows, n), out_dtype, x)
    _check(lib().grouped_gemm_bf16_int4(x.data_ptr(), ldx, q.data_ptr(), scales.data_ptr(), s_bf16, group,
                                        row_offsets.data_ptr(), act, int(gated), out.data_ptr(), ldy, code,
                                        rows, n, k, E, _stream_of(x)))
    return out


# ------------------------------------------ cross entropy of a linear head
def _head(x, w, targets):
    _dev(w, torch.bfloat16, "w")
    ldx = _rows(x, torch.bfloat16, "x")
    if w.dim() != 2 or x.shape[1] != w.shape[1] or w.shape[0] == 0:
        raise ValueError("x must be [m, k] and w [vocab, k]")
    wide = targets.dtype == torch.int64
    _dev(targets, torch.int64 if wide else torch.int32, "targets")
    if targets.shape != (x.shape[0],):
        raise ValueError("targets must be [m]")
    return ldx, int(wide), x.shape[0], w.shape[0], w.shape[1]


def linear_cross_entropy(x, w, targets, workspace=None):
    """Softmax cross entropy of each row of x w^T at its target, without the
    logits in memory: x bf16 [m, k] (rows may be strided), w bf16 [vocab, k],
    targets int64 or int32 [m] -> (loss, lse) float32 [m], lse the log of the sum
    of exponentials for the backward pass.  A target outside [0, vocab) means
    none: loss 0."""
    ldx, wide, m, vocab, k = _head(x, w, targets)
    loss, lse = x.new_empty(m, dtype=torch.float32), x.new_empty(m, dtype=torch.float32)
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        workspace, ws, ws_bytes = _workspace_of(L.fg8_linear_cross_entropy_workspace_bytes(m, vocab, k), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.linear_cross_entropy(x.data_ptr(), ldx, w.data_ptr(), targets.data_ptr(), wide, loss.data_ptr(),
                                  lse.data_ptr(), m, vocab, k, ws, ws_bytes, stream))
    return loss, lse


def linear_cross_entropy_backward(dloss, x, w, targets, lse, dw_dtype=torch.float32, needs=(True, True),
                                  workspace=None):
    """Gradients of linear_cross_entropy: dloss float32 [m] (1 / count for a mean),
    lse as the forward pass returned it -> (dx bf16 [m, k], dw dw_dtype [vocab,
    k]); `needs` leaves out (None) what is not wanted.  dx and a bfloat16 dw take
    the logits' gradients rounded to bfloat16, a float32 dw to 2^-16 (in two
    parts)."""
    ldx, wide, m, vocab, k = _head(x, w, targets)
    for name, t in (("dloss", dloss), ("lse", lse)):
        _dev(t, torch.float32, name)
        if t.shape != (m,):
            raise ValueError(f"{name} must be [m]")
    dx = x.new_empty((m, k)) if needs[0] else None
    dw = w.new_empty(w.shape, dtype=dw_dtype) if needs[1] else None
    code = _out_code(dw_dtype)
    if m == 0:     # sums over no rows
        return dx, dw if dw is None else dw.zero_()
    L = lib()
    stream = _stream_of(x)
    if workspace is None:
        # (the second part of the logits' gradients is a float dw's alone)
        workspace, ws, ws_bytes = _workspace_of(
            L.fg8_linear_cross_entropy_backward_workspace_bytes(m, vocab, k, code if needs[1] else OUT_BF16), x, stream)
    else:
        ws, ws_bytes = _workspace_given(workspace)
    _check(L.linear_cross_entropy_backward(dloss.data_ptr(), x.data_ptr(), ldx, w.data_ptr(), targets.data_ptr(), wide,
                                           lse.data_ptr(), _ptr(dx), _ptr(dw), code, m, vocab, k, ws, ws_bytes,
                                           stream))
    return dx, dw


# --------------------------------------------------------------- layer norm
def _norm_rows(t, dtype, name):
    """(rows, cols, row stride) of [..., cols]; more than two dimensions have
    to be contiguous."""
    if t.dim() != 2:
        _dev(t, dtype, name)
        cols = t.shape[-1]
        return t.numel() // cols if cols else 0, cols, cols
    ld = _rows(t, dtype, name)
    return t.shape[0], t.shape[1], ld if t.shape[0] > 1 else t.shape[1]


def _norm_dtype(x):
    return torch.bfloat16 if x.dtype == torch.bfloat16 else torch.float32


def layer_norm(x, weight, bias=None, eps=1e-5):
    """x float32 or bfloat16 [..., cols] (2-D rows may be strided), weight and
    bias both float32 or both bfloat16 [cols] -> (y of x's type and shape, mean
    and rstd float32 [...] for the backward pass)."""
    dtype = _norm_dtype(x)
    rows, cols, ldx = _norm_rows(x, dtype, "x")
    w, w_bf16 = _param(weight, cols, "weight")
    b, b_bf16 = _param(bias, cols, "bias")
    if b is not None and b_bf16 != w_bf16:
        raise TypeError("weight and bias must have one type")
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _check(lib().layer_norm(x.data_ptr(), ldx, int(dtype == torch.bfloat16), w, b, w_bf16, eps, rows,
                            cols, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream_of(x)))
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """dy and x of one type [..., cols], weight [cols], mean and rstd as
    layer_norm returned them -> (dx of x's type, dweight, dbias float32
    [cols])."""
    dtype = _norm_dtype(x)
    rows, cols, ldx = _norm_rows(x, dtype, "x")
    _, _, lddy = _norm_rows(dy, dtype, "dy")
    w, w_bf16 = _param(weight, cols, "weight")
    _dev(mean, torch.float32, "mean")
    _dev(rstd, torch.float32, "rstd")
    if dy.shape != x.shape or mean.shape != x.shape[:-1] or rstd.shape != x.shape[:-1]:
        raise ValueError("operand shapes disagree")
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    dw = x.new_empty(cols, dtype=torch.float32)
    db = torch.empty_like(dw)
    L = lib()
    bf16 = int(dtype == torch.bfloat16)
    need = L.fg8_layer_norm_backward_workspace_bytes(rows, cols, bf16)
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    _check(L.layer_norm_backward(dy.data_ptr(), lddy, x.data_ptr(), ldx, bf16, w, w_bf16,
                                 mean.data_ptr(), rstd.data_ptr(), rows, cols, dx.data_ptr(),
                                 dw.data_ptr(), db.data_ptr(), _ptr(ws), need, _stream_of(x)))
    return dx, dw, db


# -------------------------------------------------------------- MoE combine
def _combine_args(y, token_row, weights):
    dtype = _norm_dtype(y)
    _dev(y, dtype, "y")
    _dev(token_row, torch.int32, "token_row")
    _dev(weights, torch.float32, "weights")
    if y.dim() != 2 or token_row.dim() != 2 or weights.shape != token_row.shape:
        raise ValueError("y must be [rows, hidden], token_row and weights [tokens, topk]")
    return dtype, y.shape[0], y.shape[1], token_row.shape[0], token_row.shape[1]


def moe_combine(y, token_row, weights, residual=None, out=None):
    """Each token's expert rows weighted and summed: y float32 or bfloat16
    [rows, hidden], token_row int32 [tokens, topk] (as
    moe_contiguous_layout_fp8 returns it; positions outside [0, rows) add
    nothing), weights float32 [tokens, topk], residual [tokens, hidden] of y's
    type -> [tokens, hidden] of y's type."""
    dtype, rows, hidden, tokens, topk = _combine_args(y, token_row, weights)
    if out is None:
        out = y.new_empty((tokens, hidden))
    for name, t in (("residual", residual), ("out", out)):
        if t is not None:
            _dev(t, dtype, name)
            if t.shape != (tokens, hidden):
                raise ValueError(f"{name} must have shape ({tokens}, {hidden})")
    _check(lib().moe_combine(y.data_ptr(), int(dtype == torch.bfloat16), rows, token_row.data_ptr(),
                             weights.data_ptr(), _ptr(residual), tokens, topk, hidden,
                             out.data_ptr(), _stream_of(y)))
    return out


def moe_combine_backward(dout, y, token_row, row_token, weights):
    """Gradients of moe_combine (the residual's is dout itself): row_token
    int32 [rows] is token_row's inverse as moe_contiguous_layout_fp8 returns it
    -> (dy [rows, hidden] of y's type, zeros in rows that hold no token,
    dweights float32 [tokens, topk])."""
    dtype, rows, hidden, tokens, topk = _combine_args(y, token_row, weights)
    _dev(dout, dtype, "dout")
    _dev(row_token, torch.int32, "row_token")
    if dout.shape != (tokens, hidden) or row_token.shape != (rows,):
        raise ValueError("operand shapes disagree")
    dy = y.new_empty((rows, hidden))
    dweights = y.new_empty((tokens, topk), dtype=torch.float32)
    _check(lib().moe_combine_backward(dout.data_ptr(), y.data_ptr(), int(dtype == torch.bfloat16),
                                      rows, token_row.data_ptr(), row_token.data_ptr(),
                                      weights.data_ptr(), tokens, topk, hidden, dy.data_ptr(),
                                      dweights.data_ptr(), _stream_of(y)))
    return dy, dweights
