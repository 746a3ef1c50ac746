"""Python binding of libcider (include/cider.h): argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors that already live on the GPU (PyTorch is used for device memory and
the current stream, nothing else). Every step of the computation runs in the
HIP kernels of libcider.so; if the library is missing, or the device is not a
gfx950, the call raises instead of computing anything some other way.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import re
import struct
import typing

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libcider.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "cider.h")

CIDER_SUCCESS = 0
CIDER_ERROR_INVALID_VALUE = 1
CIDER_ERROR_NOT_SUPPORTED = 2
CIDER_ERROR_LAUNCH = 3
CIDER_ERROR_SCRATCH_LIMIT = 4
NOALLOC_SCRATCH_BYTES = 48 * 1024 * 1024

_c_i64, _c_i32, _c_p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p

# (restype, argtypes) of every entry point declared in include/cider.h
SIGNATURES = {
    "cider_is_available": (ctypes.c_int, []),
    "cider_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cider_version": (ctypes.c_int, []),
    "cider_quant_act": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "cider_quant_weight": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i32, _c_i32, _c_p, _c_p, _c_p]),
    "cider_w8a8_gemm": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p]),
    "cider_w4a8_gemm": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "cider_gemm_acc_i32": (ctypes.c_int, [_c_i32, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p]),
    "cider_w8a8_gemm_token_group": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p,
                                                   _c_p, _c_i64, _c_p]),
    "cider_w8a8_gemm_token_group_dt": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p,
                                                      _c_i32, _c_p, _c_i64, _c_p]),
    "cider_w8a8_gemm_split": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "cider_w8a8_gemm_split_dt": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_i32,
                                                _c_p]),
    "cider_linear_workspace_size": (ctypes.c_int64, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32]),
    "cider_gemm_workspace_size": (ctypes.c_int64, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32]),
    "cider_w8a8_gemm_ex": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_i32, _c_p,
                                         _c_i64, _c_p]),
    "cider_w8a8_gemm_noalloc": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_i32,
                                              _c_p]),
    "cider_w4a8_gemm_ex": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i32, _c_p, _c_i64,
                                         _c_p]),
    "cider_linear": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_p, _c_i64, _c_p,
                                    _c_p]),
    "cider_linear_dt": (ctypes.c_int, [_c_p, _c_i32, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_p,
                                       _c_i64, _c_p, _c_p]),
    "cider_quant_weight_clip": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i32, _c_i32, ctypes.c_double, _c_p,
                                               _c_p, _c_p]),
    "cider_quant_act_dt": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "cider_quant_weight_dt": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i32, _c_i32, _c_p, _c_p, _c_p]),
    "cider_w8a8_gemm_dt": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_i32, _c_p]),
    "cider_w4a8_gemm_dt": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i32, _c_p]),
    "cider_read_probe": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p]),
    "cider_int8_mv": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p]),
    "cider_stack_workspace_layout": (ctypes.c_int64, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i64,
                                                      ctypes.POINTER(ctypes.c_int64)]),
    "cider_stack_forward": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p, _c_p,
                                           _c_i64, _c_p, _c_p]),
    "cider_stack_forward_dt": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_i32, _c_p,
                                              _c_p, _c_i64, _c_p, _c_p]),
    "cider_moe_plan_workspace_size": (ctypes.c_int64, [_c_i64, _c_i32, _c_i32]),
    "cider_moe_plan": (ctypes.c_int, [_c_p, _c_i64, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_p]),
    **{name: (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_i32, _c_p,
                             _c_i32, _c_p])
       for name in ("cider_w8a8_grouped_gemm", "cider_w4a8_grouped_gemm", "cider_w8a8_grouped_swiglu",
                    "cider_w4a8_grouped_swiglu")},
    "cider_norm_quant": (ctypes.c_int, [_c_p, _c_p]),
    "cider_dequant_act": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_i32, _c_p]),
    "cider_rope": (ctypes.c_int, [_c_p, _c_p]),
    "cider_kv4_append": (ctypes.c_int, [_c_p, _c_p]),
    "cider_kv4_read": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p, _c_i32, _c_p]),
    "cider_kv4_attention_workspace_size": (ctypes.c_int64, [_c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i64]),
    "cider_kv4_attention": (ctypes.c_int, [_c_p, _c_p]),
}

STACK_PROJECTIONS = ("q", "k", "v", "o", "gate", "up", "down")
STACK_REGIONS = ("codes", "scales", "q", "k", "v", "o", "gate", "up", "h")


class StackLayer(ctypes.Structure):
    """cider_stack_layer_t: device pointers of one layer's 7 weight matrices."""
    _fields_ = [("w", ctypes.c_void_p * 7), ("s", ctypes.c_void_p * 7)]



class NormQuant(ctypes.Structure):
    """cider_norm_quant_t: device pointers (None leaves a part out) and sizes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "block", "slots", "weights", "post_weight", "gate", "norm_weight",
                                               "h", "normed", "x_q", "x_scale")] + \
               [(n, ctypes.c_int64) for n in ("M", "K", "block_rows", "rows_per_gate")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "top_k", "group_size")] + \
               [("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class Rope(ctypes.Structure):
    """cider_rope_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "positions", "inv_freq", "y")] + \
               [(n, ctypes.c_int64) for n in ("T", "x_row_stride", "x_head_stride", "y_row_stride", "y_head_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "heads", "head_dim", "rotary_dim", "interleaved")] + \
               [("scale", ctypes.c_float)]


class Kv4CacheArrays(ctypes.Structure):
    """cider_kv4_cache_t: the cache's device pointers and sizes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scale", "v_codes", "v_scale")] + \
               [("n_pages", ctypes.c_int64)] + \
               [(n, ctypes.c_int32) for n in ("page_size", "kv_heads", "head_dim", "group_size")]


class Kv4Append(ctypes.Structure):
    """cider_kv4_append_t (None leaves a part out)."""
    _fields_ = [("cache", Kv4CacheArrays)] + \
               [(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_norm", "k_norm", "positions", "inv_freq", "slots",
                                               "q_out")] + \
               [(n, ctypes.c_int64) for n in ("T", "q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                              "v_row_stride", "v_head_stride", "out_row_stride", "out_head_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "q_heads", "rotary_dim", "interleaved")] + \
               [("rope_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class Kv4Attention(ctypes.Structure):
    """cider_kv4_attention_t."""
    _fields_ = [("cache", Kv4CacheArrays)] + \
               [(n, ctypes.c_void_p) for n in ("q", "page_table", "lengths", "query_offsets", "y", "workspace")] + \
               [(n, ctypes.c_int64) for n in ("workspace_bytes", "T", "B", "max_pages", "q_row_stride",
                                              "q_head_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "q_heads", "causal", "window")] + \
               [("softmax_scale", ctypes.c_float)]


def _packer(cls):
    """A function that packs a structure's values, in the order of its fields
    (nested ones in place, 0 for no pointer), into bytes that a C call takes by
    address: a third of the time of filling the ctypes structure, and numbers
    that do not fit their field raise instead of being taken modulo 2^32."""
    def codes(c):
        letter = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
        return "".join(letter[t] if t in letter else codes(t) for _, t in c._fields_)
    form = struct.Struct(codes(cls))
    form = struct.Struct(f"{codes(cls)}{ctypes.sizeof(cls) - form.size}x")
    assert form.size == ctypes.sizeof(cls)

    def pack(*values):
        try:
            return form.pack(*values)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"{cls.__doc__.split()[0].rstrip('.:')}: {e}") from None
    return pack


_pack_rope, _pack_cache, _pack_append, _pack_attention = map(_packer, (Rope, Kv4CacheArrays, Kv4Append, Kv4Attention))

_lib = None


class CiderError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def header_entry_points(path: str = HEADER_PATH):
    """Names of the functions include/cider.h declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(cider_[a-z0-9_]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """Load libcider.so (built in-tree by w8a8_online_quantized_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m w8a8_online_quantized_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().cider_status_string(status).decode()


def _check(fn: str, status: int):
    if status != CIDER_SUCCESS:
        raise CiderError(fn, status, status_string(status))


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(fn):
    """Run the wrapped call with `stream` (when given) as torch's current
    stream, so that every output and temporary it allocates belongs to the
    stream its kernels run on: torch's caching allocator then reuses a freed
    temporary only for later work on that same stream, never while a kernel
    of the call may still read it."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        ctx = torch.cuda.stream(stream) if stream != torch.cuda.current_stream() else contextlib.nullcontext()
        with ctx:
            return fn(*args, stream=stream, **kw)
    return wrapper


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, shape, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _carg(a):
    """A call argument in C form: a tensor as its device pointer, a stream as
    its handle, anything else as given (ctypes converts ints and None)."""
    import torch
    if isinstance(a, torch.Tensor):
        return ctypes.c_void_p(a.data_ptr())
    if isinstance(a, torch.cuda.Stream):
        return ctypes.c_void_p(a.cuda_stream)
    return a


def prepared(fn_name: str, *args):
    """A zero-argument callable that calls the C entry point `fn_name` with
    its arguments already in C form (tensors as device pointers, the stream
    as its handle) and raises on a non-zero status. Timing loops use it so
    that back-to-back launches of short kernels are not paced by Python-side
    argument checking; the caller keeps the tensors alive."""
    f = getattr(lib(), fn_name)
    cargs = tuple(_carg(a) for a in args)

    def call():
        st = f(*cargs)
        if st != CIDER_SUCCESS:
            _check(fn_name, st)
    return call


def cider_is_available() -> bool:
    return bool(lib().cider_is_available())


def cider_version() -> int:
    return int(lib().cider_version())


CIDER_DTYPE_F16, CIDER_DTYPE_BF16 = 0, 1


def _fp_code(t, name):
    """cider_dtype_t of an fp16 / bf16 tensor."""
    import torch
    if t.dtype == torch.float16:
        return CIDER_DTYPE_F16
    if t.dtype == torch.bfloat16:
        return CIDER_DTYPE_BF16
    raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")


def _scale_shape(rows, K, group_size):
    return (rows,) if group_size == 0 else (rows, K // group_size)


@_on_stream
def cider_quant_act(x, group_size: int = 0, x_q=None, x_scale=None, stream=None):
    """fp16 or bf16 [M, K] -> (int8 codes [M, K], fp32 scales [M] or [M, K/gs])."""
    import torch
    M, K = x.shape
    dt = _fp_code(x, "x")
    _need(x, x.dtype, (M, K), "x")
    if x_q is None:
        x_q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(_scale_shape(M, K, group_size), dtype=torch.float32, device=x.device)
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(x_scale, torch.float32, _scale_shape(M, K, group_size), "x_scale")
    _check("cider_quant_act_dt", lib().cider_quant_act_dt(_ptr(x), dt, M, K, group_size, _ptr(x_q), _ptr(x_scale),
                                                          _stream(stream)))
    return x_q, x_scale


@_on_stream
def cider_quant_weight(w, bits: int = 8, group_size: int = 0, w_q=None, w_scale=None, stream=None):
    """fp16 or bf16 [N, K] -> (int8 [N, K] or packed uint8 [N, K/2], fp32 scales)."""
    import torch
    N, K = w.shape
    dt = _fp_code(w, "w")
    _need(w, w.dtype, (N, K), "w")
    qshape = (N, K) if bits == 8 else (N, K // 2)
    qdtype = torch.int8 if bits == 8 else torch.uint8
    if w_q is None:
        w_q = torch.empty(qshape, dtype=qdtype, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(_scale_shape(N, K, group_size), dtype=torch.float32, device=w.device)
    _need(w_q, qdtype, qshape, "w_q")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    _check("cider_quant_weight_dt", lib().cider_quant_weight_dt(_ptr(w), dt, N, K, bits, group_size, _ptr(w_q),
                                                                _ptr(w_scale), _stream(stream)))
    return w_q, w_scale


@_on_stream
def cider_quant_weight_clip(w, bits: int = 8, group_size: int = 0, percentile: float = 99.9, w_q=None,
                            w_scale=None, stream=None):
    """cider_quant_weight with percentile-clipped scales (same outputs)."""
    import torch
    N, K = w.shape
    dt = _fp_code(w, "w")
    _need(w, w.dtype, (N, K), "w")
    qshape = (N, K) if bits == 8 else (N, K // 2)
    qdtype = torch.int8 if bits == 8 else torch.uint8
    if w_q is None:
        w_q = torch.empty(qshape, dtype=qdtype, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(_scale_shape(N, K, group_size), dtype=torch.float32, device=w.device)
    _need(w_q, qdtype, qshape, "w_q")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    _check("cider_quant_weight_clip",
           lib().cider_quant_weight_clip(_ptr(w), dt, N, K, bits, group_size, float(percentile), _ptr(w_q),
                                         _ptr(w_scale), _stream(stream)))
    return w_q, w_scale


def cider_gemm_workspace_size(M: int, N: int, K: int, bits: int = 8, group_size: int = 0) -> int:
    """Split-K workspace bytes the GEMM dispatch uses at this shape (0: none)."""
    n = int(lib().cider_gemm_workspace_size(M, N, K, bits, group_size))
    if n < 0:
        raise ValueError("invalid GEMM sizes")
    return n


def _ws_args(workspace):
    """Pointer and bytes of a workspace, which kernels write: it must be device
    memory, and its bytes one range."""
    if workspace is None:
        return None, 0
    if not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA (HIP) tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


@_on_stream
def cider_w8a8_gemm(x_q, x_scale, w_q, w_scale, group_size: int = 0, y=None, stream=None, out_dtype=None,
                    workspace=None):
    """int8 codes + scales -> y [M, N] (fused dequant): fp16, or bf16 when
    out_dtype (or a given y) is bfloat16. A workspace of at least
    cider_gemm_workspace_size bytes enables split-K where the plan uses it."""
    import torch
    M, K = x_q.shape
    N = w_q.shape[0]
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(w_q, torch.int8, (N, K), "w_q")
    if group_size and K % group_size:
        raise ValueError("K must be a multiple of group_size")
    _need(x_scale, torch.float32, _scale_shape(M, K, group_size), "x_scale")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or torch.float16, device=x_q.device)
    dt = _fp_code(y, "y")
    _need(y, y.dtype, (M, N), "y")
    wsp, wsb = _ws_args(workspace)
    _check("cider_w8a8_gemm_ex", lib().cider_w8a8_gemm_ex(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale),
                                                          M, N, K, group_size, _ptr(y), dt, wsp, wsb,
                                                          _stream(stream)))
    return y


@_on_stream
def cider_w8a8_gemm_noalloc(x_q, x_scale, w_q, w_scale, group_size: int = 0, y=None, stream=None, out_dtype=None):
    """cider_w8a8_gemm with the split-K scratch in the library's own device
    array (the C call allocates nothing; pass y to allocate nothing here
    either). Calls that overlap in time on one GPU race on that array."""
    import torch
    M, K = x_q.shape
    N = w_q.shape[0]
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(w_q, torch.int8, (N, K), "w_q")
    if group_size and K % group_size:
        raise ValueError("K must be a multiple of group_size")
    _need(x_scale, torch.float32, _scale_shape(M, K, group_size), "x_scale")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or torch.float16, device=x_q.device)
    dt = _fp_code(y, "y")
    _need(y, y.dtype, (M, N), "y")
    _check("cider_w8a8_gemm_noalloc", lib().cider_w8a8_gemm_noalloc(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale),
                                                                    M, N, K, group_size, _ptr(y), dt, _stream(stream)))
    return y


@_on_stream
def cider_w8a8_gemm_token_group(x_q, x_scale, w_q, w_scale, group_size: int, y=None, stream=None, workspace=None,
                                out_dtype=None):
    """Per-token activation codes (x_scale [M]) times per-group weight codes
    (w_scale [N, K/group_size], group_size 64 or 128) -> y [M, N]: fp16, or
    bf16 when out_dtype (or a given y) is bfloat16."""
    import torch
    M, K = x_q.shape
    N = w_q.shape[0]
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(w_q, torch.int8, (N, K), "w_q")
    if group_size not in (64, 128) or K % group_size:
        raise ValueError("group_size must be 64 or 128 and divide K")
    _need(x_scale, torch.float32, (M,), "x_scale")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or torch.float16, device=x_q.device)
    dt = _fp_code(y, "y")
    _need(y, y.dtype, (M, N), "y")
    _check("cider_w8a8_gemm_token_group_dt",
           lib().cider_w8a8_gemm_token_group_dt(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale), M, N, K,
                                                group_size, _ptr(y), dt, *_ws_args(workspace), _stream(stream)))
    return y


@_on_stream
def cider_w8a8_gemm_split(x_q, x_scale, w_q, w_scale, part_n, ys=None, stream=None, out_dtype=None):
    """Per-channel GEMM of x_q against row-concatenated weights w_q [sum(part_n), K];
    returns one [M, part_n[i]] output per part: fp16, or bf16 when out_dtype
    (or the given ys) is bfloat16."""
    import torch
    M, K = x_q.shape
    N = w_q.shape[0]
    part_n = [int(n) for n in part_n]
    if sum(part_n) != N:
        raise ValueError("part widths must add up to the weight rows")
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(w_q, torch.int8, (N, K), "w_q")
    _need(x_scale, torch.float32, (M,), "x_scale")
    _need(w_scale, torch.float32, (N,), "w_scale")
    if ys is None:
        ys = [torch.empty((M, n), dtype=out_dtype or torch.float16, device=x_q.device) for n in part_n]
    dt = _fp_code(ys[0], "ys[0]")
    for i, (y, n) in enumerate(zip(ys, part_n)):
        _need(y, ys[0].dtype, (M, n), f"ys[{i}]")
    arr_n = (ctypes.c_int64 * len(part_n))(*part_n)
    arr_y = (ctypes.c_void_p * len(ys))(*[y.data_ptr() for y in ys])
    _check("cider_w8a8_gemm_split_dt",
           lib().cider_w8a8_gemm_split_dt(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale), M, K, len(part_n),
                                          ctypes.cast(arr_n, ctypes.c_void_p), ctypes.cast(arr_y, ctypes.c_void_p),
                                          dt, _stream(stream)))
    return ys


def cider_linear_workspace_size(M: int, N: int, K: int, bits: int = 8, group_size: int = 0) -> int:
    """Workspace bytes cider_linear needs (0: one launch, no workspace)."""
    n = int(lib().cider_linear_workspace_size(M, N, K, bits, group_size))
    if n < 0:
        raise ValueError("invalid linear sizes")
    return n


@_on_stream
def cider_linear(x, w, w_scale, bits: int = 8, group_size: int = 0, workspace=None, y=None, stream=None):
    """x [M, K] -> y [M, N] of the same dtype (fp16 or bf16) through the
    quantized linear (w: int8 codes [N, K] for bits 8, packed uint8 [N, K/2]
    for bits 4)."""
    import torch
    M, K = x.shape
    N = w.shape[0]
    dt = _fp_code(x, "x")
    _need(x, x.dtype, (M, K), "x")
    if bits == 8:
        _need(w, torch.int8, (N, K), "w")
    else:
        _need(w, torch.uint8, (N, K // 2), "w")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    need = cider_linear_workspace_size(M, N, K, bits, group_size)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _need(y, x.dtype, (M, N), "y")
    wsp, wsb = _ws_args(workspace)
    _check("cider_linear_dt", lib().cider_linear_dt(_ptr(x), dt, _ptr(w), _ptr(w_scale), M, N, K, bits, group_size,
                                                    wsp, wsb, _ptr(y), _stream(stream)))
    return y


@_on_stream
def cider_int8_mv(x, w_q, w_scale, group_size: int = 0, y=None, stream=None):
    """Decode MV: fp16 x [M, K] (M <= 4) times int8 weights dequantized on the
    fly -> fp16 y [M, N]; no activation quantization."""
    import torch
    M, K = x.shape
    N = w_q.shape[0]
    _need(x, torch.float16, (M, K), "x")
    _need(w_q, torch.int8, (N, K), "w_q")
    if group_size and K % group_size:
        raise ValueError("K must be a multiple of group_size")
    _need(w_scale, torch.float32, _scale_shape(N, K, group_size), "w_scale")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _need(y, torch.float16, (M, N), "y")
    _check("cider_int8_mv", lib().cider_int8_mv(_ptr(x), _ptr(w_q), _ptr(w_scale), M, N, K, group_size,
                                                _ptr(y), _stream(stream)))
    return y


def cider_read_probe(buf, sink, stream=None):
    """One pass over a device buffer (measurement helper: the single-launch
    read ceiling); `sink` is a small int32 device tensor."""
    import torch
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous device tensor")
    _need(sink, torch.int32, tuple(sink.shape), "sink")
    _check("cider_read_probe", lib().cider_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                                      _stream(stream)))


@_on_stream
def cider_w4a8_gemm(x_q, x_scale, w_packed, w_scale, y=None, stream=None, out_dtype=None, workspace=None):
    """int8 activation codes x packed int4 weights -> y [M, N] (fp16 or bf16)."""
    import torch
    M, K = x_q.shape
    N = w_packed.shape[0]
    _need(x_q, torch.int8, (M, K), "x_q")
    _need(w_packed, torch.uint8, (N, K // 2), "w_packed")
    _need(x_scale, torch.float32, (M,), "x_scale")
    _need(w_scale, torch.float32, (N,), "w_scale")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype or torch.float16, device=x_q.device)
    dt = _fp_code(y, "y")
    _need(y, y.dtype, (M, N), "y")
    wsp, wsb = _ws_args(workspace)
    _check("cider_w4a8_gemm_ex", lib().cider_w4a8_gemm_ex(_ptr(x_q), _ptr(x_scale), _ptr(w_packed), _ptr(w_scale),
                                                          M, N, K, _ptr(y), dt, wsp, wsb, _stream(stream)))
    return y


@_on_stream
def cider_gemm_acc_i32(mode: int, x_q, w, group_size: int = 0, acc=None, stream=None):
    """int32 accumulators of the GEMM main loop: [M, N], or [G, M, N] per group."""
    import torch
    M, K = x_q.shape
    N = w.shape[0]
    _need(x_q, torch.int8, (M, K), "x_q")
    if mode == 0:
        _need(w, torch.int8, (N, K), "w")
    else:
        _need(w, torch.uint8, (N, K // 2), "w")
    shape = (M, N) if group_size == 0 else (K // group_size, M, N)
    if acc is None:
        acc = torch.empty(shape, dtype=torch.int32, device=x_q.device)
    _need(acc, torch.int32, shape, "acc")
    _check("cider_gemm_acc_i32", lib().cider_gemm_acc_i32(mode, _ptr(x_q), _ptr(w), M, N, K, group_size,
                                                          _ptr(acc), _stream(stream)))
    return acc


@_on_stream
def w8a8_linear(x, w_q, w_scale, group_size: int = 0, stream=None):
    """The README's per-channel / per-group linear: quantize x, then the fused
    GEMM; the output has x's type (fp16 or bf16)."""
    x_q, x_scale = cider_quant_act(x, group_size, stream=stream)
    return cider_w8a8_gemm(x_q, x_scale, w_q, w_scale, group_size, stream=stream, out_dtype=x.dtype)


@_on_stream
def w8a8_linear_token_group(x, w_q, w_scale, group_size: int, stream=None):
    """Per-token activation quantization, then the per-group-weight GEMM."""
    x_q, x_scale = cider_quant_act(x, 0, stream=stream)
    return cider_w8a8_gemm_token_group(x_q, x_scale, w_q, w_scale, group_size, stream=stream)


@_on_stream
def w4a8_linear(x, w_packed, w_scale, stream=None):
    """The README's W4A8 linear: per-token int8 activations times packed int4
    weights; the output has x's type (fp16 or bf16)."""
    x_q, x_scale = cider_quant_act(x, 0, stream=stream)
    return cider_w4a8_gemm(x_q, x_scale, w_packed, w_scale, stream=stream, out_dtype=x.dtype)


# ---- expert blocks ----------------------------------------------------------
# A decode step runs these on a few rows, where the call costs more than its
# kernel: tensors that fit are passed with one test each, pointers go to
# ctypes as plain integers, and outputs are made in the forms that torch parses
# fastest (sizes as arguments 1.25 us, as a tuple 1.6, empty_like 1.1).

def _need_on(dev, t, dtype, shape, name):
    """_need, and that the tensor lives on the current device `dev`, where the
    call's kernels run."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return
    except AttributeError:
        pass                                        # not a tensor: _need says so
    _need(t, dtype, shape, name)
    raise ValueError(f"{name} must be on the current device {dev}, not {t.get_device()}")


def _raw_stream(stream, dev):
    import torch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_I32 = 1 << 31


def cider_moe_plan_workspace_size(T: int, top_k: int, n_experts: int) -> int:
    """Workspace bytes cider_moe_plan needs (0: one launch, no workspace)."""
    if not (-_I32 <= top_k < _I32 and -_I32 <= n_experts < _I32):
        raise ValueError("invalid routing sizes")   # (ctypes would take them modulo 2^32)
    n = lib().cider_moe_plan_workspace_size(T, top_k, n_experts)
    if n < 0:
        raise ValueError("invalid routing sizes")
    return n


_plan_workspace_size = functools.lru_cache(maxsize=256)(cider_moe_plan_workspace_size)


@_on_stream
def cider_moe_plan(expert_ids, n_experts: int, offsets=None, rows=None, slots=None, workspace=None, stream=None):
    """int32 expert ids [T, top_k] (outside [0, n_experts): no expert) ->
    (offsets [n_experts + 1], rows [T * top_k], slots [T, top_k]), all int32."""
    import torch
    dev = torch.cuda.current_device()
    T, top_k = shape = expert_ids.shape
    _need_on(dev, expert_ids, torch.int32, shape, "expert_ids")
    need = _plan_workspace_size(T, top_k, n_experts)
    if offsets is None:
        offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=expert_ids.device)
    else:
        _need_on(dev, offsets, torch.int32, (n_experts + 1,), "offsets")
    if rows is None:
        rows = torch.empty(T * top_k, dtype=torch.int32, device=expert_ids.device)
    else:
        _need_on(dev, rows, torch.int32, (T * top_k,), "rows")
    if slots is None:
        slots = torch.empty_like(expert_ids)
    else:
        _need_on(dev, slots, torch.int32, shape, "slots")
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=expert_ids.device)
    elif workspace is not None and workspace.is_cuda and workspace.get_device() != dev:
        raise ValueError(f"workspace must be on the current device {dev}, not {workspace.get_device()}")
    st = lib().cider_moe_plan(expert_ids.data_ptr(), T, top_k, n_experts, offsets.data_ptr(), rows.data_ptr(),
                              slots.data_ptr(), *_ws_args(workspace), _raw_stream(stream, dev))
    if st:
        _check("cider_moe_plan", st)
    return offsets, rows, slots


def _grouped(fn, gated, bits, x_q, x_scale, w, w_scale, offsets, row_index, row_div, y, stream, out_dtype):
    import torch
    dev = torch.cuda.current_device()
    x_rows, K = x_q.shape
    E, N = w_scale.shape
    _need_on(dev, x_q, torch.int8, (x_rows, K), "x_q")
    _need_on(dev, x_scale, torch.float32, (x_rows,), "x_scale")
    if bits == 8:
        _need_on(dev, w, torch.int8, (E, N, K), "w_q")
    else:
        _need_on(dev, w, torch.uint8, (E, N, K // 2), "w_packed")
    _need_on(dev, w_scale, torch.float32, (E, N), "w_scale")
    _need_on(dev, offsets, torch.int32, (E + 1,), "offsets")
    P, index = x_rows, None
    if row_index is not None:
        P, index = row_index.numel(), row_index.data_ptr()
        _need_on(dev, row_index, torch.int32, (P,), "row_index")
    if not -_I32 <= row_div < _I32:
        raise ValueError("row_div must be from 1 to 2^31 - 1")   # (ctypes would take it modulo 2^32)
    if gated and N % 2:
        raise ValueError("the gated product needs as many gate rows as up rows")
    n_out = N // 2 if gated else N
    if y is None:
        y = torch.empty(P, n_out, dtype=out_dtype or torch.float16, device=x_q.device)
    else:
        _need_on(dev, y, y.dtype, (P, n_out), "y")
    st = getattr(lib(), fn)(x_q.data_ptr(), x_scale.data_ptr(), x_rows, w.data_ptr(), w_scale.data_ptr(),
                            offsets.data_ptr(), index, row_div, P, N, K, E, y.data_ptr(), _fp_code(y, "y"),
                            _raw_stream(stream, dev))
    if st:
        _check(fn, st)
    return y


@_on_stream
def cider_w8a8_grouped_gemm(x_q, x_scale, w_q, w_scale, offsets, row_index=None, row_div: int = 1, y=None, stream=None,
                            out_dtype=None):
    """Products grouped by expert: rows offsets[e] .. offsets[e+1] - 1 of y
    [P, N] (fp16, or bf16 when out_dtype or a given y is) are activation rows
    row_index[p] // row_div (p without an index) times expert e's int8 weights
    w_q [E, N, K]. offsets int32 [E + 1] on the GPU; rows past its last value
    are left as they were."""
    return _grouped("cider_w8a8_grouped_gemm", False, 8, x_q, x_scale, w_q, w_scale, offsets, row_index, row_div, y,
                    stream, out_dtype)


@_on_stream
def cider_w4a8_grouped_gemm(x_q, x_scale, w_packed, w_scale, offsets, row_index=None, row_div: int = 1, y=None,
                            stream=None, out_dtype=None):
    """cider_w8a8_grouped_gemm with packed int4 weights [E, N, K / 2], K below 131072."""
    return _grouped("cider_w4a8_grouped_gemm", False, 4, x_q, x_scale, w_packed, w_scale, offsets, row_index, row_div,
                    y, stream, out_dtype)


@_on_stream
def cider_w8a8_grouped_swiglu(x_q, x_scale, w_q, w_scale, offsets, row_index=None, row_div: int = 1, y=None,
                              stream=None, out_dtype=None):
    """The grouped product with the gated activation: weight rows 0 .. N/2 - 1
    of an expert are gates and the others ups, y [P, N/2] = silu(gate) * up."""
    return _grouped("cider_w8a8_grouped_swiglu", True, 8, x_q, x_scale, w_q, w_scale, offsets, row_index, row_div, y,
                    stream, out_dtype)


@_on_stream
def cider_w4a8_grouped_swiglu(x_q, x_scale, w_packed, w_scale, offsets, row_index=None, row_div: int = 1, y=None,
                              stream=None, out_dtype=None):
    """cider_w8a8_grouped_swiglu with packed int4 weights [E, N, K / 2], K below 131072."""
    return _grouped("cider_w4a8_grouped_swiglu", True, 4, x_q, x_scale, w_packed, w_scale, offsets, row_index, row_div,
                    y, stream, out_dtype)


@_on_stream
def cider_norm_quant(x=None, block=None, norm_weight=None, slots=None, weights=None, post_weight=None, gate=None,
                     rows_per_gate: int = 0, alpha: float = 1.0, eps: float = 1e-6, group_size: int = 0, h=None,
                     normed=None, x_q=None, x_scale=None, stream=None):
    """The boundary between two blocks -> (h, x_q, x_scale):
    h = x + alpha * gate * post_norm(block), codes of norm(h). x [M, K] and
    block [M, K] (or expert rows [R, K] summed by slots and weights [M, top_k])
    fp16 or bf16; see cider_norm_quant in include/cider.h. Without block, h is
    x itself; without norm_weight there are no codes (None, None). `normed`, a
    tensor [M, K], also receives the unquantized norm; h may be x (in place)."""
    import torch
    dev = torch.cuda.current_device()
    fp = x if x is not None else block
    if fp is None:
        raise ValueError("x or block must be given")
    K, t = fp.shape[1], fp.dtype
    M = fp.shape[0] if x is not None or slots is None else slots.shape[0]
    if group_size and K % group_size:
        raise ValueError("K must be a multiple of group_size")
    row, vec = (M, K), (K,)
    top_k = block_rows = 0
    px = pb = ps = pw = pp = pg = pn = ph = pd = pq = pc = None
    if x is not None:
        _need_on(dev, x, t, row, "x")
        px = x.data_ptr()
    if slots is not None:
        if block is None:
            raise ValueError("slots need a block")
        top_k, block_rows = slots.shape[1], block.shape[0]
        _need_on(dev, slots, torch.int32, (M, top_k), "slots")
        _need_on(dev, weights, torch.float32, (M, top_k), "weights")
        ps, pw = slots.data_ptr(), weights.data_ptr()
    elif weights is not None:
        raise ValueError("weights need slots")
    if block is not None:
        _need_on(dev, block, t, (block_rows, K) if slots is not None else row, "block")
        pb = block.data_ptr()
        if h is None:
            h = torch.empty(M, K, dtype=t, device=fp.device) if x is None else torch.empty_like(x)
    if post_weight is not None:
        _need_on(dev, post_weight, t, vec, "post_weight")
        pp = post_weight.data_ptr()
    if gate is not None:
        if rows_per_gate < 0:
            raise ValueError("rows_per_gate must not be negative")
        one = rows_per_gate == 0 and gate.dim() == 1
        _need_on(dev, gate, t, vec if one else (-(-M // rows_per_gate) if rows_per_gate else 1, K), "gate")
        pg = gate.data_ptr()
    if h is not None:
        _need_on(dev, h, t, row, "h")
        ph = h.data_ptr()
        if slots is not None and not block_rows:
            pb = ph                                 # no expert rows: nothing is read, and an empty tensor has no pointer
    if normed is not None:
        _need_on(dev, normed, t, row, "normed")
        pd = normed.data_ptr()
    if norm_weight is not None:
        _need_on(dev, norm_weight, t, vec, "norm_weight")
        pn = norm_weight.data_ptr()
        scales = _scale_shape(M, K, group_size)
        if x_q is None:
            x_q = torch.empty(M, K, dtype=torch.int8, device=fp.device)
        else:
            _need_on(dev, x_q, torch.int8, row, "x_q")
        if x_scale is None:
            x_scale = torch.empty(*scales, dtype=torch.float32, device=fp.device)
        else:
            _need_on(dev, x_scale, torch.float32, scales, "x_scale")
        pq, pc = x_q.data_ptr(), x_scale.data_ptr()
    elif x_q is not None or x_scale is not None:
        raise ValueError("codes need a norm_weight")
    args = NormQuant(px, pb, ps, pw, pp, pg, pn, ph, pd, pq, pc, M, K, block_rows, rows_per_gate, _fp_code(fp, "x"),
                     top_k, group_size, alpha, eps)
    st = lib().cider_norm_quant(ctypes.byref(args), _raw_stream(stream, dev))
    if st:
        _check("cider_norm_quant", st)
    return (h if h is not None else x), x_q, x_scale


@_on_stream
def cider_dequant_act(x_q, x_scale, group_size: int = 0, y=None, stream=None, out_dtype=None):
    """int8 codes [M, K] and their scales -> rows [M, K], fp16 or (out_dtype or
    a given y) bf16: what the quantized linears take them to be."""
    import torch
    dev = torch.cuda.current_device()
    M, K = row = x_q.shape
    _need_on(dev, x_q, torch.int8, row, "x_q")
    if group_size and K % group_size:
        raise ValueError("K must be a multiple of group_size")
    _need_on(dev, x_scale, torch.float32, _scale_shape(M, K, group_size), "x_scale")
    if y is None:
        y = torch.empty(M, K, dtype=out_dtype or torch.float16, device=x_q.device)
    else:
        _need_on(dev, y, y.dtype, row, "y")
    st = lib().cider_dequant_act(x_q.data_ptr(), x_scale.data_ptr(), M, K, group_size, y.data_ptr(), _fp_code(y, "y"),
                                 _raw_stream(stream, dev))
    if st:
        _check("cider_dequant_act", st)
    return y


@_on_stream
def w8a8_moe(x_q, x_scale, expert_ids, gate_up, gate_up_scale, down, down_scale, out_dtype=None, stream=None):
    """The experts of a block on the tokens' codes (from cider_norm_quant or
    cider_quant_act): gate_up int8 [E, 2I, K] or packed uint8 [E, 2I, K/2],
    down [E, N, I] likewise. Returns (expert rows [T * top_k, N], slots), which
    cider_norm_quant sums into the residual. Ids of no expert have slot -1, and
    as many of the last expert rows hold nothing that was written."""
    import torch
    t = out_dtype or torch.float16
    top_k, E = expert_ids.shape[1], gate_up.shape[0]
    offsets, rows, slots = cider_moe_plan(expert_ids, E, stream=stream)
    up_call = cider_w8a8_grouped_swiglu if gate_up.dtype == torch.int8 else cider_w4a8_grouped_swiglu
    down_call = cider_w8a8_grouped_gemm if down.dtype == torch.int8 else cider_w4a8_grouped_gemm
    a = up_call(x_q, x_scale, gate_up, gate_up_scale, offsets, row_index=rows, row_div=top_k, out_dtype=t,
                stream=stream)
    a_q, a_scale = cider_quant_act(a, 0, stream=stream)
    return down_call(a_q, a_scale, down, down_scale, offsets, out_dtype=t, stream=stream), slots


# ---- attention blocks -------------------------------------------------------

class KV4Cache(typing.NamedTuple):
    """A paged cache of keys and values in 4 bits (cider_kv4_cache_t in
    include/cider.h): k_codes, v_codes uint8 [n_pages, kv_heads, page_size,
    head_dim / 2], k_scale, v_scale fp32 [n_pages, kv_heads, G, page_size]."""
    k_codes: typing.Any
    k_scale: typing.Any
    v_codes: typing.Any
    v_scale: typing.Any


def kv4_cache(n_pages: int, kv_heads: int, page_size: int, head_dim: int, group_size: int = 0, device=None) -> KV4Cache:
    """An empty KV4Cache (codes 0, scales 0) on the current device. group_size 0
    gives one scale per token and head, 32 or more one per group of dimensions
    (head_dim, or a half or a quarter of it)."""
    import torch
    if group_size and (group_size < 32 or group_size not in (head_dim, head_dim / 2, head_dim / 4)):
        raise ValueError(f"group_size must be 0, or head_dim, head_dim / 2 or head_dim / 4 and at least 32, got {group_size}")
    G = head_dim // group_size if group_size else 1
    device = device or torch.device("cuda", torch.cuda.current_device())
    codes, scale = (n_pages, kv_heads, page_size, head_dim // 2), (n_pages, kv_heads, G, page_size)
    return KV4Cache(torch.full(codes, 0x88, dtype=torch.uint8, device=device), torch.zeros(scale, device=device),
                    torch.full(codes, 0x88, dtype=torch.uint8, device=device), torch.zeros(scale, device=device))


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     trained: int = 8192, fast: float = 32.0, slow: float = 1.0, device=None):
    """(inv_freq fp64 [rotary_dim / 2] on the GPU, scale) for cider_rope and
    cider_kv4_append: base^(-2i/rotary_dim), scaled for contexts `factor` times
    the `trained` length:

    * None: as they are;
    * "linear": divided by factor (positions interpolated);
    * "base": base times factor^(d / (d - 2)), so that the slowest pair turns
      factor times slower and the fastest as before;
    * "parts": pairs that turn less than `slow` times over the trained length
      divided by factor, those that turn more than `fast` times as they are, a
      ramp between, and scale 0.1 ln(factor) + 1 (Peng et al., YaRN, 2023)."""
    import torch
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not factor >= 1.0 or not base > 1.0 or not math.isfinite(base * factor):
        raise ValueError("factor must be at least 1 and base above 1")
    d, scale = rotary_dim, 1.0
    if scaling == "base":
        base = base * factor ** (d / (d - 2)) if d > 2 else base
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "parts":
        if trained < 1 or not fast > slow > 0:
            raise ValueError("parts need a trained length and fast > slow > 0")
        pair = lambda turns: d * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), d - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(d // 2)]
        freq = [f / factor * r + f * (1.0 - r) for f, r in zip(freq, ramp)]
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    device = device or torch.device("cuda", torch.cuda.current_device())
    return torch.tensor(freq, dtype=torch.float64, device=device), scale


def _need_rows(dev, t, dtype, shape, name):
    """A [T, heads, D] tensor on the current device whose heads are contiguous:
    its (row, head) strides. A dimension of one has a stride of its own."""
    import torch
    try:
        fits = t.dtype is dtype and t.shape == shape and t.get_device() == dev
    except AttributeError:
        fits = False
    if not fits:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be on the current device {dev}, not {t.get_device()}")
    T, H, D = shape
    row, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name} must have contiguous heads")
    if H == 1:
        head = D
    return (row if T > 1 else H * D), head


def _refused(fn, status, cache=None, **tensors):
    """Raise for a call that returned a status, and say which tensors start at
    no multiple of 16 bytes, as slices like slots[1:] may: of all that these
    calls refuse, what a tensor's type and shape do not show."""
    if status == CIDER_ERROR_INVALID_VALUE:
        if cache is not None:
            tensors.update(cache._asdict() if isinstance(cache, KV4Cache) else zip(KV4Cache._fields, cache))
        off = [name for name, t in tensors.items() if t is not None and t.data_ptr() % 16]
        if off:
            raise CiderError(fn, status, f"{status_string(status)}: {', '.join(off)} must start at a multiple of 16 bytes "
                                         "(a slice's copy does)")
    _check(fn, status)


def _cache_args(dev, cache):
    """The values of cider_kv4_cache_t."""
    import torch
    k_codes, k_scale, v_codes, v_scale = cache
    n_pages, hkv, page, half = codes = k_codes.shape
    G = k_scale.shape[2]
    scales = (n_pages, hkv, G, page)
    _need_on(dev, k_codes, torch.uint8, codes, "k_codes")
    _need_on(dev, v_codes, torch.uint8, codes, "v_codes")
    _need_on(dev, k_scale, torch.float32, scales, "k_scale")
    _need_on(dev, v_scale, torch.float32, scales, "v_scale")
    D = 2 * half
    if not G or D % G:
        raise ValueError("the cache's groups must divide its heads")
    return (k_codes.data_ptr(), k_scale.data_ptr(), v_codes.data_ptr(), v_scale.data_ptr(), n_pages, page, hkv, D, D // G)


def _rotation(dev, T, positions, inv_freq):
    import torch
    n = inv_freq.numel()
    _need_on(dev, positions, torch.int32, (T,), "positions")
    _need_on(dev, inv_freq, torch.float64, (n,), "inv_freq")
    return positions.data_ptr(), inv_freq.data_ptr(), 2 * n


@_on_stream
def cider_rope(x, positions, inv_freq, interleaved: bool = False, scale: float = 1.0, y=None, stream=None):
    """Rotary positions: x [T, heads, D] (fp16 or bf16, heads contiguous) with
    the first 2 * len(inv_freq) dimensions of each head turned by positions
    (int32 [T]) times inv_freq (fp64) -> y, x's shape, contiguous unless given
    (y may be x). See cider_rope in include/cider.h; rope_frequencies makes
    inv_freq and scale."""
    import torch
    dev = torch.cuda.current_device()
    T, H, D = shape = x.shape
    t = x.dtype
    xr, xh = _need_rows(dev, x, t, shape, "x")
    pos, freq, rd = _rotation(dev, T, positions, inv_freq)
    if y is None:
        y, yr, yh = torch.empty(T, H, D, dtype=t, device=x.device), H * D, D
    else:
        yr, yh = _need_rows(dev, y, t, shape, "y")
    args = _pack_rope(x.data_ptr(), pos, freq, y.data_ptr(), T, xr, xh, yr, yh, _fp_code(x, "x"), H, D, rd,
                      1 if interleaved else 0, scale)
    st = lib().cider_rope(args, _raw_stream(stream, dev))
    if st:
        _refused("cider_rope", st, x=x, positions=positions, inv_freq=inv_freq, y=y)
    return y


@_on_stream
def cider_kv4_append(cache, k, v, slots, q=None, positions=None, inv_freq=None, interleaved: bool = False,
                     rope_scale: float = 1.0, q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None, stream=None):
    """New tokens' k, v [T, kv_heads, D] into a KV4Cache at slots (int32 [T],
    page * page_size + offset; outside the cache: not stored), after k's head
    norm (k_norm [D]) and rotation (positions, inv_freq), where given. q [T,
    q_heads, D] goes through q_norm and the rotation to q_out, which is
    returned (contiguous unless given; it may be q). See cider_kv4_append in
    include/cider.h. The slots of a call must differ."""
    import torch
    dev = torch.cuda.current_device()
    arrays = _cache_args(dev, cache)
    T, Hkv, D, t = k.shape[0], arrays[6], arrays[7], k.dtype
    rows = (T, Hkv, D)
    kr, kh = _need_rows(dev, k, t, rows, "k")
    vr, vh = _need_rows(dev, v, t, rows, "v")
    _need_on(dev, slots, torch.int32, (T,), "slots")
    pq = pqn = pkn = pos = freq = po = 0
    qr = qh = our = ouh = Hq = rd = 0
    if q is not None:
        Hq = q.shape[1]
        rows = (T, Hq, D)
        qr, qh = _need_rows(dev, q, t, rows, "q")
        if q_out is None:
            q_out, our, ouh = torch.empty(T, Hq, D, dtype=t, device=q.device), Hq * D, D
        else:
            our, ouh = _need_rows(dev, q_out, t, rows, "q_out")
        pq, po = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm need q")
    if q_norm is not None:
        _need_on(dev, q_norm, t, (D,), "q_norm")
        pqn = q_norm.data_ptr()
    if k_norm is not None:
        _need_on(dev, k_norm, t, (D,), "k_norm")
        pkn = k_norm.data_ptr()
    if positions is not None:
        if inv_freq is None:
            raise ValueError("positions need inv_freq")
        pos, freq, rd = _rotation(dev, T, positions, inv_freq)
    elif inv_freq is not None:
        raise ValueError("inv_freq needs positions")
    args = _pack_append(*arrays, pq, k.data_ptr(), v.data_ptr(), pqn, pkn, pos, freq, slots.data_ptr(), po, T, qr, qh, kr,
                        kh, vr, vh, our, ouh, _fp_code(k, "k"), Hq, rd, 1 if interleaved else 0, rope_scale, eps)
    st = lib().cider_kv4_append(args, _raw_stream(stream, dev))
    if st:
        _refused("cider_kv4_append", st, cache, k=k, v=v, slots=slots, q=q, positions=positions, inv_freq=inv_freq,
                 q_norm=q_norm, k_norm=k_norm, q_out=q_out)
    return q_out


@_on_stream
def cider_kv4_read(cache, slots, k=None, v=None, stream=None, out_dtype=None):
    """The cache's rows at slots (int32 [n]) -> (k, v) [n, kv_heads, D], fp16 or
    (out_dtype or a given k) bf16; zeros for slots outside the cache."""
    import torch
    dev = torch.cuda.current_device()
    arrays = _cache_args(dev, cache)
    n = slots.numel()
    shape = (n, arrays[6], arrays[7])
    _need_on(dev, slots, torch.int32, (n,), "slots")
    if k is None:
        k = torch.empty(*shape, dtype=out_dtype or (v.dtype if v is not None else torch.float16), device=slots.device)
    else:
        _need_on(dev, k, k.dtype, shape, "k")
    if v is None:
        v = torch.empty_like(k)
    else:
        _need_on(dev, v, k.dtype, shape, "v")
    st = lib().cider_kv4_read(_pack_cache(*arrays), slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _fp_code(k, "k"),
                              _raw_stream(stream, dev))
    if st:
        _refused("cider_kv4_read", st, cache, slots=slots, k=k, v=v)
    return k, v


def cider_kv4_attention_workspace_size(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int, capacity: int) -> int:
    """Workspace bytes cider_kv4_attention needs for T query rows of B sequences
    whose page tables hold `capacity` tokens (0: one launch, no workspace)."""
    if not all(-_I32 <= n < _I32 for n in (q_heads, kv_heads, head_dim)):
        raise ValueError("invalid attention sizes")   # (ctypes would take them modulo 2^32)
    n = lib().cider_kv4_attention_workspace_size(T, B, q_heads, kv_heads, head_dim, capacity)
    if n < 0:
        raise ValueError("invalid attention sizes")
    return n


_attention_workspace_size = functools.lru_cache(maxsize=256)(cider_kv4_attention_workspace_size)


@_on_stream
def cider_kv4_attention(q, cache, page_table, lengths, query_offsets=None, causal: bool = True, window: int = 0,
                        softmax_scale: float | None = None, y=None, workspace=None, stream=None):
    """Attention of q [T, q_heads, D] (fp16 or bf16) over a KV4Cache -> y [T,
    q_heads, D]. page_table int32 [B, max_pages], lengths int32 [B] (tokens in
    the cache, those of the queries included), query_offsets int32 [B + 1] (or
    T / B query rows per sequence), all on the GPU. Queries stand at the end of
    their sequences; with causal each sees the tokens up to its own, with a
    window only the last `window` of them. softmax_scale is D^-0.5 if not
    given. See cider_kv4_attention in include/cider.h."""
    import torch
    dev = torch.cuda.current_device()
    arrays = _cache_args(dev, cache)
    T, Hq, D = shape = q.shape
    t = q.dtype
    if D != arrays[7]:
        raise ValueError(f"q must have heads of {arrays[7]}, got {D}")
    qr, qh = _need_rows(dev, q, t, shape, "q")
    B, max_pages = pages = page_table.shape
    _need_on(dev, page_table, torch.int32, pages, "page_table")
    _need_on(dev, lengths, torch.int32, (B,), "lengths")
    offsets = 0
    if query_offsets is not None:
        _need_on(dev, query_offsets, torch.int32, (B + 1,), "query_offsets")
        offsets = query_offsets.data_ptr()
    if window < 0:
        raise ValueError("window must not be negative")
    if y is None:
        y = torch.empty(T, Hq, D, dtype=t, device=q.device)
    else:
        _need_on(dev, y, t, shape, "y")
    space, size = 0, _attention_workspace_size(T, B, Hq, arrays[6], D, max_pages * arrays[5])
    if workspace is not None:
        _, size = _ws_args(workspace)
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be on the current device {dev}, not {workspace.get_device()}")
    elif size:
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        space = workspace.data_ptr()
    args = _pack_attention(*arrays, q.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), offsets, y.data_ptr(), space, size,
                           T, B, max_pages, qr, qh, _fp_code(q, "q"), Hq, 1 if causal else 0, min(window, _I32 - 1),
                           D ** -0.5 if softmax_scale is None else softmax_scale)
    st = lib().cider_kv4_attention(args, _raw_stream(stream, dev))
    if st:
        _refused("cider_kv4_attention", st, cache, q=q, page_table=page_table, lengths=lengths, query_offsets=query_offsets,
                 y=y, workspace=workspace)
    return y


@_on_stream
def w8a8_attention(x_q, x_scale, w_qkv, qkv_scale, w_out, out_scale, cache, slots, page_table, lengths, q_heads: int,
                   query_offsets=None, positions=None, inv_freq=None, interleaved: bool = False, rope_scale: float = 1.0,
                   q_norm=None, k_norm=None, eps: float = 1e-6, causal: bool = True, window: int = 0,
                   softmax_scale: float | None = None, out_dtype=None, stream=None):
    """The attention of a block on the tokens' codes (from cider_norm_quant or
    cider_quant_act): w_qkv int8 [(q_heads + 2 kv_heads) * D, K], w_out [N,
    q_heads * D], both with fp32 scales per row. The tokens' keys and values go
    into the cache at `slots`, lengths count them, and the result [T, N] is the
    block's output, which cider_norm_quant adds to the residual."""
    import torch
    t = out_dtype or torch.float16
    T, Hkv, D = x_q.shape[0], cache.k_codes.shape[1], 2 * cache.k_codes.shape[3]
    q, k, v = cider_w8a8_gemm_split(x_q, x_scale, w_qkv, qkv_scale, [q_heads * D, Hkv * D, Hkv * D], stream=stream,
                                    out_dtype=t)
    q = q.view(T, q_heads, D)
    cider_kv4_append(cache, k.view(T, Hkv, D), v.view(T, Hkv, D), slots, q=q, positions=positions, inv_freq=inv_freq,
                     interleaved=interleaved, rope_scale=rope_scale, q_norm=q_norm, k_norm=k_norm, eps=eps, q_out=q,
                     stream=stream)
    a = cider_kv4_attention(q, cache, page_table, lengths, query_offsets=query_offsets, causal=causal, window=window,
                            softmax_scale=softmax_scale, stream=stream)
    a_q, a_scale = cider_quant_act(a.view(T, q_heads * D), 0, stream=stream)
    return cider_w8a8_gemm(a_q, a_scale, w_out, out_scale, 0, stream=stream, out_dtype=t)


def cider_stack_workspace_layout(M: int, hidden: int, q_dim: int, kv_dim: int, mlp_dim: int):
    """(total bytes, {region: byte offset}) of the stack driver's workspace."""
    offs = (ctypes.c_int64 * 9)()
    total = int(lib().cider_stack_workspace_layout(M, hidden, q_dim, kv_dim, mlp_dim, offs))
    return total, dict(zip(STACK_REGIONS, list(offs)))


def stack_region(workspace, offsets, name, M, hidden, q_dim, kv_dim, mlp_dim, dtype=None):
    """A torch view of one workspace region (for checking intermediates);
    dtype: torch.float16 (default) or torch.bfloat16 for a bf16 chain."""
    import torch
    dims = {"q": q_dim, "k": kv_dim, "v": kv_dim, "o": hidden, "gate": mlp_dim, "up": mlp_dim, "h": hidden}
    n = dims[name]
    start = offsets[name]
    return workspace[start:start + 2 * M * n].view(dtype or torch.float16).view(M, n)


def fuse_stack_layer(layer):
    """A copy of one stack layer ({name: (codes, scales)}) whose q/k/v and
    gate/up codes and scales live back to back in one allocation each, so
    that cider_stack_forward runs each group as one GEMM."""
    import torch
    out = dict(layer)
    for group in (("q", "k", "v"), ("gate", "up")):
        wcat = torch.cat([layer[n][0] for n in group])
        scat = torch.cat([layer[n][1] for n in group])
        r = 0
        for n in group:
            rows = layer[n][0].shape[0]
            out[n] = (wcat[r:r + rows], scat[r:r + rows])
            r += rows
    return out


@_on_stream
def cider_stack_forward(x, layers, dims, workspace=None, y=None, stream=None):
    """Runs the chained linear stack. `layers`: list of dicts {name: (codes, scales)}
    for the seven projections; dims = (hidden, q_dim, kv_dim, mlp_dim)."""
    import torch
    hidden, q_dim, kv_dim, mlp_dim = dims
    M = x.shape[0]
    dt = _fp_code(x, "x")
    _need(x, x.dtype, (M, hidden), "x")
    total, _ = cider_stack_workspace_layout(M, hidden, q_dim, kv_dim, mlp_dim)
    if workspace is None:
        workspace = torch.empty(total, dtype=torch.uint8, device=x.device)
    if y is None:
        y = torch.empty((M, hidden), dtype=x.dtype, device=x.device)
    _need(y, x.dtype, (M, hidden), "y")
    arr = (StackLayer * len(layers))()
    for i, L in enumerate(layers):
        for j, name in enumerate(STACK_PROJECTIONS):
            wq, ws = L[name]
            arr[i].w[j] = wq.data_ptr()
            arr[i].s[j] = ws.data_ptr()
    _check("cider_stack_forward_dt", lib().cider_stack_forward_dt(
        _ptr(x), dt, M, hidden, q_dim, kv_dim, mlp_dim, len(layers), ctypes.cast(arr, ctypes.c_void_p),
        *_ws_args(workspace), _ptr(y), _stream(stream)))
    return y, workspace
