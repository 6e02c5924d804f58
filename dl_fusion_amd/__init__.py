"""Python binding of libdlfusion, the fused Conv/MatMul -> BatchNorm -> activation
operator for MI355X (gfx950).

This module only marshals arguments to the C ABI declared in
``include/dlfusion.h`` (same function names).  Every step of the operator runs
in the library's HIP kernels or its host fold; there is no Python or CPU
fallback: importing fails loudly when ``libdlfusion.so`` has not been built.

Device buffers are passed as contiguous torch tensors (their ``data_ptr()``)
or as raw integer addresses; host buffers of the fold functions are numpy
arrays.  ``stream=None`` means torch's current stream on the current device.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# DLF_LIBRARY names another build of the same library (the sanitizer build of the host code the
# CPU test-suite runs under); by default the in-tree build
LIB_PATH = os.environ.get("DLF_LIBRARY") or os.path.join(_HERE, "libdlfusion.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first (python -c 'import __graft_entry__ as g; g.build()')")

# torch's ROCm build carries its own HIP runtime under the same soname as the system one the
# library links against.  Loading torch first makes the library bind to that runtime, so one
# HIP runtime serves the process; with the library loaded first, its calls found no device
# while torch's allocations went on working.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------------------
# Enums and descriptors (mirror include/dlfusion.h)
# ---------------------------------------------------------------------------
DLF_OK, DLF_ERR_INVALID_ARG, DLF_ERR_UNSUPPORTED, DLF_ERR_HIP, DLF_ERR_ALIAS = 0, -1, -2, -3, -4
DLF_F32, DLF_BF16, DLF_FP8_E4M3 = 0, 1, 2
DLF_ACT_NONE, DLF_ACT_RELU, DLF_ACT_GELU_TANH, DLF_ACT_GELU_ERF = 0, 1, 2, 3

DTYPES = {"f32": DLF_F32, "bf16": DLF_BF16, "fp8": DLF_FP8_E4M3}
ACTS = {"none": DLF_ACT_NONE, "relu": DLF_ACT_RELU, "gelu_tanh": DLF_ACT_GELU_TANH, "gelu_erf": DLF_ACT_GELU_ERF}
DLF_GATE_SILU, DLF_GATE_GELU_TANH, DLF_GATE_GELU_ERF = 0, 1, 2
GATES = {"silu": DLF_GATE_SILU, "gelu_tanh": DLF_GATE_GELU_TANH, "gelu_erf": DLF_GATE_GELU_ERF}


class dlf_conv_desc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("w", ctypes.c_int64),
                ("c_in", ctypes.c_int64), ("c_out", ctypes.c_int64), ("kh", ctypes.c_int64),
                ("kw", ctypes.c_int64), ("stride_h", ctypes.c_int32), ("stride_w", ctypes.c_int32),
                ("pad_h", ctypes.c_int32), ("pad_w", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int)]


class dlf_gemm_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("act", ctypes.c_int),
                ("out_inv_scale", ctypes.c_float)]


def conv_desc(n, h, w, c_in, c_out, kh=3, kw=3, stride=1, pad=1, dtype="bf16", act="relu"):
    return dlf_conv_desc(n, h, w, c_in, c_out, kh, kw, stride, stride, pad, pad,
                         DTYPES.get(dtype, dtype), ACTS.get(act, act))


def gemm_desc(m, n, k, in_dtype="bf16", out_dtype="bf16", act="none", out_inv_scale=1.0):
    return dlf_gemm_desc(m, n, k, DTYPES.get(in_dtype, in_dtype), DTYPES.get(out_dtype, out_dtype),
                         ACTS.get(act, act), out_inv_scale)


OPS = {"input": 0, "conv": 1, "matmul": 2, "matmul_fp8": 3, "bias_add": 4, "batchnorm": 5, "add": 6,
       "relu": 7, "gelu": 8, "gelu_erf": 9, "quant": 10}
DLF_OP_OTHER = 11
DLF_NODE_OUTPUT, DLF_NODE_TRAINING = 1, 2


class dlf_ffn_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("d_model", ctypes.c_int64), ("d_ff", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int)]


def ffn_desc(m, d_model, d_ff, act="gelu_tanh", dtype="bf16"):
    return dlf_ffn_desc(m, d_model, d_ff, DTYPES.get(dtype, dtype), ACTS.get(act, act))


class dlf_kv_cache_desc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


def kv_cache_desc(pages, kv_heads, page_size, head_dim, dtype="bf16", k_scale=1.0, v_scale=1.0):
    return dlf_kv_cache_desc(pages, kv_heads, page_size, head_dim, DTYPES.get(dtype, dtype), k_scale, v_scale)


class dlf_page_plan_desc(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("token_cap", ctypes.c_int32), ("free_cap", ctypes.c_int32)]


def page_plan_desc(requests, page_size, max_pages, token_cap, free_cap):
    return dlf_page_plan_desc(requests, page_size, max_pages, token_cap, free_cap)


class dlf_paged_attn_desc(ctypes.Structure):
    _fields_ = [("cache", dlf_kv_cache_desc), ("requests", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("window", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("softmax_scale", ctypes.c_float)]


def paged_attn_desc(cache, requests, heads, max_pages, softmax_scale, window=0, max_len=0, q_stride=None):
    return dlf_paged_attn_desc(cache, requests, heads, max_pages, window, max_len,
                               heads * cache.head_dim if q_stride is None else q_stride, softmax_scale)


class dlf_lora_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("adapters", ctypes.c_int32), ("requests", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("base_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("dtype", ctypes.c_int)]


def lora_desc(m, n, k, rank, adapters, requests=0, x_stride=None, base_stride=None, out_stride=None, dtype="bf16"):
    return dlf_lora_desc(m, n, k, rank, adapters, requests, k if x_stride is None else x_stride,
                         n if base_stride is None else base_stride, n if out_stride is None else out_stride,
                         DTYPES.get(dtype, dtype))


DLF_SCALE_BLOCK = 128


def scale_stride(cols):
    """Floats between two rows of block scales that lie close: one a 128 columns, rounded up to a multiple of 4."""
    return -(-cols // (4 * DLF_SCALE_BLOCK)) * 4


class dlf_rms_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("scale_stride", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("sum_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("out_inv_scale", ctypes.c_float)]


def rms_norm_desc(rows, cols, eps=1e-5, dtype="bf16", out_dtype="bf16", out_inv_scale=1.0, x_stride=None,
                  residual_stride=None, sum_stride=None, y_stride=None, y_scale_stride=None):
    strides = [cols if s is None else s for s in (x_stride, residual_stride, sum_stride, y_stride)]
    return dlf_rms_norm_desc(rows, cols, scale_stride(cols) if y_scale_stride is None else y_scale_stride, *strides,
                             DTYPES.get(dtype, dtype), DTYPES.get(out_dtype, out_dtype), eps, out_inv_scale)


class dlf_quant_blocks_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("scale_stride", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("codes_stride", ctypes.c_int64), ("dtype", ctypes.c_int)]


def quant_blocks_desc(rows, cols, dtype="bf16", x_stride=None, codes_stride=None, row_scale_stride=None):
    return dlf_quant_blocks_desc(rows, cols, scale_stride(cols) if row_scale_stride is None else row_scale_stride,
                                 cols if x_stride is None else x_stride,
                                 cols if codes_stride is None else codes_stride, DTYPES.get(dtype, dtype))


class dlf_gemm_blocks_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("a_scale_stride", ctypes.c_int32), ("b_scale_stride", ctypes.c_int32), ("act", ctypes.c_int)]


def gemm_blocks_desc(m, n, k, act="none", a_scale_stride=None, b_scale_stride=None):
    close = scale_stride(k)
    return dlf_gemm_blocks_desc(m, n, k, close if a_scale_stride is None else a_scale_stride,
                                close if b_scale_stride is None else b_scale_stride, ACTS.get(act, act))


class dlf_graph_node(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32), ("n_inputs", ctypes.c_int32), ("inputs", ctypes.c_int32 * 2),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("rank", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("shape", ctypes.c_int64 * 4), ("flops", ctypes.c_int64)]


class dlf_fusion_group(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("nodes", ctypes.c_int32 * 5), ("saved_bytes", ctypes.c_int64),
                ("net_benefit", ctypes.c_double)]


_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_f32p = ctypes.POINTER(ctypes.c_float)
_SIGS = {
    "dlf_fold_bn": [_i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_double, ctypes.c_int, _vp, _vp],
    "dlf_bn_scale_shift": [_i64, _vp, _vp, _vp, _vp, _vp, ctypes.c_double, ctypes.c_double, _vp, _vp],
    "dlf_conv_fused": [ctypes.POINTER(dlf_conv_desc), _vp, _vp, _vp, _vp, _vp, _vp],
    "dlf_gemm_fused": [ctypes.POINTER(dlf_gemm_desc), _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "dlf_gemm_fused_split": [ctypes.POINTER(dlf_gemm_desc), _vp, _vp, _vp, _vp, ctypes.c_int32,
                             ctypes.POINTER(_vp), _vp],
    "dlf_gemm_fused_gated": [ctypes.POINTER(dlf_gemm_desc), _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp],
    "dlf_conv_plain": [ctypes.POINTER(dlf_conv_desc), _vp, _vp, _vp, _vp, _vp],
    "dlf_gemm_plain": [ctypes.POINTER(dlf_gemm_desc), _vp, _vp, ctypes.c_float, _vp, _vp],
    "dlf_bn_apply": [_i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, ctypes.c_double, _vp, _vp],
    "dlf_scale_shift_apply": [_i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp],
    "dlf_add": [_i64, ctypes.c_int, _vp, _vp, _vp, _vp],
    "dlf_act_apply": [_i64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp],
    "dlf_quant_apply": [_i64, _vp, ctypes.c_float, _vp, _vp],
    "dlf_ffn_pack": [_i64, _i64, _vp, _vp],
    "dlf_ffn_fused": [ctypes.POINTER(dlf_ffn_desc), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "dlf_ffn_workspace_bytes": [ctypes.POINTER(dlf_ffn_desc), ctypes.POINTER(ctypes.c_size_t)],
    "dlf_ffn_fused_ws": [ctypes.POINTER(dlf_ffn_desc), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                         _vp],
    "dlf_ffn_fused_noalloc": [ctypes.POINTER(dlf_ffn_desc), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "dlf_page_plan": [ctypes.POINTER(dlf_page_plan_desc)] + [_vp] * 11,
    "dlf_paged_store": [ctypes.POINTER(dlf_kv_cache_desc), _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp],
    "dlf_paged_attention_workspace_bytes": [ctypes.POINTER(dlf_paged_attn_desc), ctypes.POINTER(ctypes.c_size_t)],
    "dlf_paged_attention": [ctypes.POINTER(dlf_paged_attn_desc)] + [_vp] * 8 + [ctypes.c_size_t, _vp],
    "dlf_lora_workspace_bytes": [ctypes.POINTER(dlf_lora_desc), ctypes.POINTER(ctypes.c_size_t)],
    "dlf_lora_add": [ctypes.POINTER(dlf_lora_desc)] + [_vp] * 9 + [ctypes.c_size_t, _vp],
    "dlf_rms_norm": [ctypes.POINTER(dlf_rms_norm_desc)] + [_vp] * 7,
    "dlf_quant_blocks": [ctypes.POINTER(dlf_quant_blocks_desc)] + [_vp] * 4,
    "dlf_gemm_blocks_workspace_bytes": [ctypes.POINTER(dlf_gemm_blocks_desc), ctypes.POINTER(ctypes.c_size_t)],
    "dlf_gemm_blocks": [ctypes.POINTER(dlf_gemm_blocks_desc)] + [_vp] * 8 + [ctypes.c_size_t, _vp],
    "dlf_gemm_blocks_gated": [ctypes.POINTER(dlf_gemm_blocks_desc)] + [_vp] * 5 + [ctypes.c_int, _vp, _vp,
                                                                                   ctypes.c_size_t, _vp],
    "dlf_quant_blocks_weights": [_i64, _i64, _vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp],
    "dlf_clock_probe": [ctypes.c_int32, ctypes.c_int32, _vp, _vp],
    "dlf_fusion_plan": [ctypes.POINTER(dlf_graph_node), ctypes.c_int32, ctypes.c_double, ctypes.c_double,
                        ctypes.POINTER(dlf_fusion_group), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = ctypes.c_int
    _fn.argtypes = _args
_lib.dlf_status_string.restype = ctypes.c_char_p
_lib.dlf_status_string.argtypes = [ctypes.c_int]
_lib.dlf_last_error.restype = ctypes.c_char_p
_lib.dlf_last_error.argtypes = []
_lib.dlf_tuning_reload.restype = None
_lib.dlf_tuning_reload.argtypes = []


class DlfError(RuntimeError):
    def __init__(self, status: int, func: str):
        self.status = status
        self.detail = dlf_last_error()
        super().__init__(f"{func}: {dlf_status_string(status)}: {self.detail}")


def dlf_status_string(status: int) -> str:
    return _lib.dlf_status_string(int(status)).decode()


def dlf_last_error() -> str:
    return _lib.dlf_last_error().decode()


def dlf_tuning_reload():
    """Re-read the DLF_* tuning switches from the environment (the library reads them once,
    when it is loaded)."""
    _lib.dlf_tuning_reload()


def _check(status: int, func: str):
    if status != DLF_OK:
        raise DlfError(status, func)


def _dev(t):
    """Device pointer of a contiguous torch tensor, a raw int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("device tensors must be contiguous")
    return t.data_ptr()


def _host(a, dtype=None):
    if a is None:
        return None, None
    arr = np.ascontiguousarray(a, dtype=dtype) if dtype is not None else np.ascontiguousarray(a)
    return arr, arr.ctypes.data


def _stream(stream):
    if stream is None:
        # the handle itself: torch.cuda.current_stream() builds a Stream object around it, which took
        # 2.7 us of a call's 8.5 on the host; this takes 0.2
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# Host-side fold
# ---------------------------------------------------------------------------
def dlf_fold_bn(w, conv_bias, gamma, beta, mean, var, eps, w_out_dtype="bf16"):
    """Fold BN into conv weights (host, binary64, one RNE rounding).  w is fp32
    [cout, ...] (OHWI); returns (w_out [same shape] as float32 or uint16 bf16 bits,
    bias_out float32 [cout])."""
    w_arr, w_p = _host(w, np.float32)
    cout = w_arr.shape[0] if w_arr.ndim else 0
    k = w_arr.size // cout if cout else 0
    dt = DTYPES.get(w_out_dtype, w_out_dtype)
    out = np.empty(w_arr.shape, dtype=np.float32 if dt == DLF_F32 else np.uint16)
    bias_out = np.empty(cout, dtype=np.float32)
    keep = [_host(v, np.float32) for v in (conv_bias, gamma, beta, mean, var)]
    st = _lib.dlf_fold_bn(cout, k, w_p, *[p for _, p in keep], float(eps), dt, out.ctypes.data,
                          bias_out.ctypes.data)
    _check(st, "dlf_fold_bn")
    return out, bias_out


def dlf_bn_scale_shift(conv_bias, gamma, beta, mean, var, eps, pre_scale=1.0):
    """Per-channel (alpha, beta') with BN(acc * pre_scale + b) = acc * alpha + beta' (host)."""
    g, _ = _host(gamma, np.float32)
    cout = g.size
    scale = np.empty(cout, dtype=np.float32)
    shift = np.empty(cout, dtype=np.float32)
    keep = [_host(v, np.float32) for v in (conv_bias, gamma, beta, mean, var)]
    st = _lib.dlf_bn_scale_shift(cout, *[p for _, p in keep], float(eps), float(pre_scale),
                                 scale.ctypes.data, shift.ctypes.data)
    _check(st, "dlf_bn_scale_shift")
    return scale, shift


# ---------------------------------------------------------------------------
# Device entry points (asynchronous on `stream`)
# ---------------------------------------------------------------------------
def dlf_conv_fused(desc, x, w, bias, residual, y, stream=None):
    _check(_lib.dlf_conv_fused(ctypes.byref(desc), _dev(x), _dev(w), _dev(bias), _dev(residual), _dev(y),
                               _stream(stream)), "dlf_conv_fused")


def dlf_gemm_fused(desc, a, b, col_scale, col_shift, residual, c, stream=None):
    _check(_lib.dlf_gemm_fused(ctypes.byref(desc), _dev(a), _dev(b), _dev(col_scale), _dev(col_shift),
                               _dev(residual), _dev(c), _stream(stream)), "dlf_gemm_fused")


def dlf_gemm_fused_gated(desc, a, b, col_scale, col_shift, gate, c, stream=None):
    """Gated projection: c[:, j] = gate(g_j) * u_j over interleaved (gate, up) weight rows."""
    _check(_lib.dlf_gemm_fused_gated(ctypes.byref(desc), _dev(a), _dev(b), _dev(col_scale), _dev(col_shift),
                                     GATES.get(gate, gate), _dev(c), _stream(stream)), "dlf_gemm_fused_gated")


def dlf_gemm_fused_split(desc, a, b, col_scale, col_shift, outs, stream=None):
    """One GEMM, its columns stored to len(outs) tensors (see include/dlfusion.h)."""
    arr = (_vp * max(1, len(outs)))(*[_dev(o) for o in outs])
    _check(_lib.dlf_gemm_fused_split(ctypes.byref(desc), _dev(a), _dev(b), _dev(col_scale), _dev(col_shift),
                                     len(outs), arr, _stream(stream)), "dlf_gemm_fused_split")


def dlf_conv_plain(desc, x, w, conv_bias, y, stream=None):
    _check(_lib.dlf_conv_plain(ctypes.byref(desc), _dev(x), _dev(w), _dev(conv_bias), _dev(y), _stream(stream)),
           "dlf_conv_plain")


def dlf_gemm_plain(desc, a, b, dequant, y, stream=None):
    _check(_lib.dlf_gemm_plain(ctypes.byref(desc), _dev(a), _dev(b), float(dequant), _dev(y), _stream(stream)),
           "dlf_gemm_plain")


def dlf_bn_apply(rows, c, dt, y, gamma, beta, mean, var, eps, z, stream=None):
    _check(_lib.dlf_bn_apply(rows, c, DTYPES.get(dt, dt), _dev(y), _dev(gamma), _dev(beta), _dev(mean), _dev(var),
                             float(eps), _dev(z), _stream(stream)), "dlf_bn_apply")


def dlf_scale_shift_apply(rows, c, dt, y, scale, shift, z, stream=None):
    _check(_lib.dlf_scale_shift_apply(rows, c, DTYPES.get(dt, dt), _dev(y), _dev(scale), _dev(shift), _dev(z),
                                      _stream(stream)), "dlf_scale_shift_apply")


def dlf_add(count, dt, a, b, out, stream=None):
    _check(_lib.dlf_add(count, DTYPES.get(dt, dt), _dev(a), _dev(b), _dev(out), _stream(stream)), "dlf_add")


def dlf_act_apply(count, dt, act, x, out, stream=None):
    _check(_lib.dlf_act_apply(count, DTYPES.get(dt, dt), ACTS.get(act, act), _dev(x), _dev(out),
                              _stream(stream)), "dlf_act_apply")


def dlf_quant_apply(count, x, inv_scale, codes, stream=None):
    _check(_lib.dlf_quant_apply(count, _dev(x), float(inv_scale), _dev(codes), _stream(stream)),
           "dlf_quant_apply")


def dlf_ffn_pack(w_bits):
    """Host: a [rows][k] bf16 weight (uint16 bit patterns) packed in the fused FFN kernel's
    fragment order; returns a new uint16 array of the same shape."""
    w, _ = _host(w_bits, np.uint16)
    out = np.empty_like(w)
    rows, k = w.shape
    _check(_lib.dlf_ffn_pack(rows, k, w.ctypes.data, out.ctypes.data), "dlf_ffn_pack")
    return out


def dlf_ffn_fused(desc, x, w1_packed, b1, w2_packed, b2, residual, y, stream=None):
    _check(_lib.dlf_ffn_fused(ctypes.byref(desc), _dev(x), _dev(w1_packed), _dev(b1), _dev(w2_packed), _dev(b2),
                              _dev(residual), _dev(y), _stream(stream)), "dlf_ffn_fused")


def dlf_ffn_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(_lib.dlf_ffn_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)), "dlf_ffn_workspace_bytes")
    return n.value


def dlf_ffn_fused_ws(desc, x, w1_packed, b1, w2_packed, b2, residual, y, workspace, workspace_bytes, stream=None):
    _check(_lib.dlf_ffn_fused_ws(ctypes.byref(desc), _dev(x), _dev(w1_packed), _dev(b1), _dev(w2_packed), _dev(b2),
                                 _dev(residual), _dev(y), _dev(workspace), int(workspace_bytes), _stream(stream)),
           "dlf_ffn_fused_ws")


DLF_FFN_NOALLOC_SCRATCH_BYTES = 32 << 20


def dlf_ffn_fused_noalloc(desc, x, w1_packed, b1, w2_packed, b2, residual, y, stream=None):
    """dlf_ffn_fused_ws without a workspace: the split's partial sums use the library's static
    device scratch (see include/dlfusion.h)."""
    _check(_lib.dlf_ffn_fused_noalloc(ctypes.byref(desc), _dev(x), _dev(w1_packed), _dev(b1), _dev(w2_packed),
                                      _dev(b2), _dev(residual), _dev(y), _stream(stream)), "dlf_ffn_fused_noalloc")


# What the operators of a decode step take for a type beside itself: its bits
_I32, _I64, _F32, _BF16, _FP8 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float8_e4m3fn
_BITS = {_BF16: (torch.int16, torch.uint16), _FP8: (torch.uint8, torch.int8)}


def _refuse(t, dtype, size, name):
    if t.dtype is not dtype and t.dtype not in _BITS.get(dtype, ()):
        raise ValueError(f"{name} has type {t.dtype}, {dtype} is needed")
    if t.nbytes < size:
        raise ValueError(f"{name} has {t.nbytes} bytes, {size} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _sized(t, dtype, size, name):
    """Device pointer of a contiguous torch tensor of ``dtype`` and at least ``size`` bytes, or a raw address
    or None as it is: these operators read indices out of their arrays, so a short one or one of another type
    would be read out of range.  Type and size take 0.05 to 0.1 us an array."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not dtype or t.nbytes < size or not t.is_contiguous():
        _refuse(t, dtype, size, name)
    return t.data_ptr()


def _table(t, rows, cols):
    """The same of a block table, whose rows are as long as the descriptor says."""
    size = 4 * rows * cols
    if t is not None and not isinstance(t, int) and t.nbytes != size and t.dim() > 1 and t.shape[-1] != cols:
        raise ValueError(f"block_table has {t.shape[-1]} columns, max_pages is {cols}")
    return _sized(t, _I32, size, "block_table")


def _workspace(t, size):
    if t is None or isinstance(t, int):
        return t
    if t.nbytes < size or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous, of at least {size} bytes")
    return t.data_ptr()


def _caches(cache, k_cache, v_cache):
    dtype, size = (_FP8, 1) if cache.dtype == DLF_FP8_E4M3 else (_BF16, 2)
    size *= cache.pages * cache.kv_heads * cache.page_size * cache.head_dim
    return _sized(k_cache, dtype, size, "k_cache"), _sized(v_cache, dtype, size, "v_cache")


def _rows(t, rank, name):
    """(device pointer, elements between rows) of a bf16 torch tensor whose dimensions after the first
    are contiguous: [rows][...] with `rank` dimensions, 2 or 3; the first may have any stride."""
    shape, strides = t.shape, t.stride()
    if len(strides) != rank:
        raise ValueError(f"{name} needs {rank} dimensions, got {len(strides)}")
    if t.dtype is not _BF16 and t.dtype not in _BITS[_BF16]:
        raise ValueError(f"{name} has type {t.dtype}, bf16 is needed")
    width = shape[-1]
    if strides[-1] != 1 and width != 1:
        raise ValueError("the dimensions after the first must be contiguous")
    if rank == 3:
        if strides[1] != width and shape[1] != 1:
            raise ValueError("the dimensions after the first must be contiguous")
        width *= shape[1]
    return t.data_ptr(), strides[0] if shape[0] > 1 else width


def dlf_page_plan(desc, cached, fresh, free_pages, free_head, block_table, starts, lens, slots, rows, counts,
                  stream=None):
    """Block tables and slot maps of a step, from the requests' lengths (see include/dlfusion.h)."""
    n, cap = desc.requests, desc.token_cap
    _check(_lib.dlf_page_plan(ctypes.byref(desc), _sized(cached, _I32, 4 * n, "cached"),
                              _sized(fresh, _I32, 4 * n, "fresh"),
                              _sized(free_pages, _I32, 4 * desc.free_cap, "free_pages"),
                              _sized(free_head, _I32, 4, "free_head"), _table(block_table, n, desc.max_pages),
                              _sized(starts, _I32, 4 * n + 4, "starts"), _sized(lens, _I32, 4 * n, "lens"),
                              _sized(slots, _I64, 8 * cap, "slots"), _sized(rows, _I32, 4 * cap, "rows"),
                              _sized(counts, _I32, 16, "counts"), _stream(stream)), "dlf_page_plan")


def dlf_paged_store(cache, k, v, slots, k_cache, v_cache, stream=None):
    """New keys and values [tokens][kv_heads][head_dim] into the cache's slots; the rows of k and v
    may be any distance apart (column blocks of a fused QKV product)."""
    kp, ks = _rows(k, 3, "k")
    vp, vs = _rows(v, 3, "v")
    tokens = k.shape[0]
    if k.shape != v.shape or k.shape[1:] != (cache.kv_heads, cache.head_dim) or slots.shape[0] != tokens:
        raise ValueError("k and v must be [tokens][kv_heads][head_dim], slots [tokens]")
    _check(_lib.dlf_paged_store(ctypes.byref(cache), tokens, kp, ks, vp, vs, _sized(slots, _I64, 8 * tokens, "slots"),
                                *_caches(cache, k_cache, v_cache), _stream(stream)), "dlf_paged_store")


def dlf_paged_attention_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(_lib.dlf_paged_attention_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)),
           "dlf_paged_attention_workspace_bytes")
    return n.value


def dlf_paged_attention(desc, q, k_cache, v_cache, block_table, lens, out, lse, workspace, workspace_bytes,
                        stream=None):
    """Attention of one new token per request over the paged cache.  q is [requests][heads][head_dim]
    with its requests desc.q_stride elements apart (a column block of a fused QKV product)."""
    n, heads, cache = desc.requests, desc.heads, desc.cache
    dim = cache.head_dim
    if isinstance(q, int):
        qp = q
    else:
        qp, qs = _rows(q, 3, "q")
        if q.shape != (n, heads, dim) or (n > 1 and qs != desc.q_stride):
            raise ValueError("q must be [requests][heads][head_dim], its requests q_stride elements apart")
    workspace_bytes = int(workspace_bytes)
    _check(_lib.dlf_paged_attention(ctypes.byref(desc), qp, *_caches(cache, k_cache, v_cache),
                                    _table(block_table, n, desc.max_pages), _sized(lens, _I32, 4 * n, "lens"),
                                    _sized(out, _BF16, 2 * n * heads * dim, "out"),
                                    _sized(lse, _F32, 4 * n * heads, "lse"), _workspace(workspace, workspace_bytes),
                                    workspace_bytes, _stream(stream)), "dlf_paged_attention")


def dlf_lora_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(_lib.dlf_lora_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)), "dlf_lora_workspace_bytes")
    return n.value


def _matrix(t, rows, cols, stride, name):
    """Device pointer of a bf16 [rows][cols] tensor whose rows are `stride` elements apart, or of a raw
    address or None as it is."""
    if t is None or isinstance(t, int):
        return t
    p, s = _rows(t, 2, name)
    if t.shape[0] != rows or t.shape[1] != cols or (rows > 1 and s != stride):
        raise ValueError(f"{name} must be [{rows}][{cols}] with rows {stride} elements apart")
    return p


def dlf_lora_add(desc, x, a, b, scale, ids, row_map, base, out, workspace, workspace_bytes, stream=None):
    """out = base + scale (x A^T) B^T by each row's own adapter (see include/dlfusion.h); the rows of
    x, base and out lie the descriptor's strides apart."""
    m, n, k, count = desc.m, desc.n, desc.k, desc.adapters
    weights = 2 * count * desc.rank
    workspace_bytes = int(workspace_bytes)
    _check(_lib.dlf_lora_add(ctypes.byref(desc), _matrix(x, m, k, desc.x_stride, "x"),
                             _sized(a, _BF16, weights * k, "a"), _sized(b, _BF16, weights * n, "b"),
                             _sized(scale, _F32, 4 * count, "scale"),
                             _sized(ids, _I32, 4 * (m if row_map is None else desc.requests), "ids"),
                             _sized(row_map, _I32, 4 * m, "row_map"), _matrix(base, m, n, desc.base_stride, "base"),
                             _matrix(out, m, n, desc.out_stride, "out"), _workspace(workspace, workspace_bytes),
                             workspace_bytes, _stream(stream)), "dlf_lora_add")


_TYPES = {DLF_F32: _F32, DLF_BF16: _BF16, DLF_FP8_E4M3: _FP8}


def _strided(t, dtype, shape, stride, name):
    """Device pointer of a tensor of the type and shape (rows, columns) that the descriptor says, its rows `stride`
    elements apart, or of a raw address or None as it is.  0.4 us a tensor where it is just that."""
    if t is None or t.__class__ is int:
        return t
    if t.shape != shape or t.dtype is not dtype or not (t.is_contiguous() if stride == shape[1] else t.stride() == (stride, 1)):
        _refuse_strided(t, dtype, shape, stride, name)
    return t.data_ptr()


def _refuse_strided(t, dtype, shape, stride, name):
    # an unknown type is the library's to refuse; the strides of a single row or column are not used
    if dtype is not None and t.dtype is not dtype and t.dtype not in _BITS.get(dtype, ()):
        raise ValueError(f"{name} has type {t.dtype}, {dtype} is needed")
    rows, cols = shape
    got = t.stride()
    if tuple(t.shape) != shape or (cols > 1 and rows > 0 and got[1] != 1) or (rows > 1 and cols > 0 and got[0] != stride):
        raise ValueError(f"{name} must be [{rows}][{cols}] with rows {stride} elements apart")


def _handle(stream, names, *tensors):
    """The stream's handle.  All tensors have to be on its device, the current one's where it is None: a kernel would fault
    on the host's or another device's memory.  A raw handle does not say whose it is: the first tensor's device.  0.5 us for
    six tensors."""
    at = -2                     # no device's: the host is -1
    for t in tensors:
        if t is not None and t.__class__ is not int:
            on = t.get_device()
            if on != at:
                if on < 0 or at >= 0:
                    _refuse_device(names, tensors, at)
                at = on
    if stream is None:
        here = torch._C._cuda_getDevice() if at >= 0 else torch.cuda.current_device()
    elif stream.__class__ is int:
        return stream
    else:
        here = stream.device.index
    if at >= 0 and at != here:
        _refuse_device(names, tensors, here)
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _refuse_device(names, tensors, here):
    for name, t in zip(names, tensors):
        if t is not None and t.__class__ is not int and (t.get_device() < 0 or t.get_device() != here):
            raise ValueError(f"{name} is on {t.device}, the call runs on " + (f"cuda:{here}" if here >= 0 else "a GPU"))


def _scales(t, rows, stride, name):
    """Device pointer of contiguous fp32 block scales [rows][stride], or of a raw address or None as it is."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not _F32 or t.nbytes < 4 * rows * stride or not t.is_contiguous():
        _refuse(t, _F32, 4 * rows * stride, name)
    return t.data_ptr()


def dlf_rms_norm(desc, x, residual, weight, sum, y, y_scale, stream=None):
    """y = norm(x + residual) * weight, and the sum itself (see include/dlfusion.h); the rows lie the descriptor's
    strides apart."""
    n, cols = shape = desc.rows, desc.cols
    dtype = _TYPES.get(desc.dtype)
    _check(_lib.dlf_rms_norm(ctypes.byref(desc), _strided(x, dtype, shape, desc.x_stride, "x"),
                             residual if residual is None else _strided(residual, dtype, shape, desc.residual_stride, "residual"),
                             _scales(weight, 1, cols, "weight"),
                             sum if sum is None else _strided(sum, dtype, shape, desc.sum_stride, "sum"),
                             _strided(y, _TYPES.get(desc.out_dtype), shape, desc.y_stride, "y"),
                             y_scale if y_scale is None else _scales(y_scale, n, desc.scale_stride, "y_scale"),
                             _handle(stream, ("x", "residual", "weight", "sum", "y", "y_scale"), x, residual, weight, sum, y,
                                     y_scale)), "dlf_rms_norm")


def dlf_quant_blocks(desc, x, codes, scale, stream=None):
    """Rows as e4m3 codes and a scale for each 128 columns (see include/dlfusion.h)."""
    shape = desc.rows, desc.cols
    _check(_lib.dlf_quant_blocks(ctypes.byref(desc), _strided(x, _TYPES.get(desc.dtype), shape, desc.x_stride, "x"),
                                 _strided(codes, _FP8, shape, desc.codes_stride, "codes"),
                                 _scales(scale, shape[0], desc.scale_stride, "scale"),
                                 _handle(stream, ("x", "codes", "scale"), x, codes, scale)), "dlf_quant_blocks")


def dlf_gemm_blocks_workspace_bytes(desc):
    n = ctypes.c_size_t(0)
    _check(_lib.dlf_gemm_blocks_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)), "dlf_gemm_blocks_workspace_bytes")
    return n.value


_GEMM_BLOCKS = ("a", "a_scale", "b", "b_scale", "col_shift", "c", "workspace", "residual")


def dlf_gemm_blocks(desc, a, a_scale, b, b_scale, col_shift, residual, c, workspace, workspace_bytes, stream=None):
    """Product of e4m3 matrices whose rows have a scale for each 128 values of k, b's for each 128 rows
    (see include/dlfusion.h)."""
    m, n, k = desc.m, desc.n, desc.k
    shape = (m, n)
    workspace_bytes = int(workspace_bytes)
    _check(_lib.dlf_gemm_blocks(ctypes.byref(desc), _strided(a, _FP8, (m, k), k, "a"),
                                _scales(a_scale, m, desc.a_scale_stride, "a_scale"), _strided(b, _FP8, (n, k), k, "b"),
                                _scales(b_scale, -(-n // 128), desc.b_scale_stride, "b_scale"),
                                col_shift if col_shift is None else _scales(col_shift, 1, n, "col_shift"),
                                residual if residual is None else _strided(residual, _BF16, shape, n, "residual"),
                                _strided(c, _BF16, shape, n, "c"), _workspace(workspace, workspace_bytes),
                                workspace_bytes, _handle(stream, _GEMM_BLOCKS, a, a_scale, b, b_scale, col_shift, c,
                                                         workspace if workspace_bytes else None, residual)), "dlf_gemm_blocks")


def dlf_gemm_blocks_gated(desc, a, a_scale, b, b_scale, col_shift, gate, c, workspace, workspace_bytes, stream=None):
    """The same with interleaved gate and up rows: c[:, j] = gate(g_j) * u_j."""
    m, n, k = desc.m, desc.n, desc.k
    workspace_bytes = int(workspace_bytes)
    _check(_lib.dlf_gemm_blocks_gated(ctypes.byref(desc), _strided(a, _FP8, (m, k), k, "a"),
                                      _scales(a_scale, m, desc.a_scale_stride, "a_scale"),
                                      _strided(b, _FP8, (n, k), k, "b"),
                                      _scales(b_scale, 2 * -(-n // 256), desc.b_scale_stride, "b_scale"),
                                      col_shift if col_shift is None else _scales(col_shift, 1, n, "col_shift"),
                                      GATES.get(gate, gate), _strided(c, _BF16, (m, n // 2), n // 2, "c"),
                                      _workspace(workspace, workspace_bytes), workspace_bytes,
                                      _handle(stream, _GEMM_BLOCKS, a, a_scale, b, b_scale, col_shift, c,
                                              workspace if workspace_bytes else None)),
           "dlf_gemm_blocks_gated")


def dlf_quant_blocks_weights(w, gated=False):
    """Host: fp32 weights [n][k] as e4m3 codes (uint8 [n][k]) and the scales of their 128 x 128 blocks (float32
    [rows][scale_stride(k)]); gated: rows 2j and 2j + 1 are gate and up (see include/dlfusion.h)."""
    arr, p = _host(w, np.float32)
    n, k = arr.shape
    stride = scale_stride(k)
    codes = np.empty((n, k), dtype=np.uint8)
    scale = np.empty((2 * -(-n // 256) if gated else -(-n // 128), stride), dtype=np.float32)
    _check(_lib.dlf_quant_blocks_weights(n, k, p, int(gated), stride, codes.ctypes.data, scale.ctypes.data),
           "dlf_quant_blocks_weights")
    return codes, scale


class Buffers(dict):
    """Tensors by name that a block keeps between calls and drops for larger ones.  The allocator knows the stream they were
    made on only, and would hand them out there again while kernels on another stream still use them: each call says that it
    uses them on its stream, and they come free when what that stream has been given by then is done."""

    def __init__(self, **tensors):
        super().__init__(tensors)
        self._gpu = all(t.is_cuda for t in self.values())
        self._told = set()

    def used(self):
        """The current stream uses all of them.  0.4 us where it has said so before."""
        if not self._gpu:
            return self
        device = torch.cuda.current_device()
        key = device, torch._C._cuda_getCurrentRawStream(device)        # default streams of all devices have one handle
        if key not in self._told:
            stream = torch.cuda.current_stream(device)
            for t in self.values():
                t.record_stream(stream)
            self._told.add(key)
        return self


def dlf_clock_probe(workgroups, iters, stamps, stream=None):
    """Enqueue the shader-clock probe; stamps: a device int64 tensor of 4 * workgroups values."""
    _check(_lib.dlf_clock_probe(int(workgroups), int(iters), _dev(stamps), _stream(stream)), "dlf_clock_probe")


def graph_nodes(graph):
    """A graph given as node dicts (op, inputs, shape, dtype, flops, output, training; op names
    as in OPS, any other name is DLF_OP_OTHER) as a dlf_graph_node array."""
    arr = (dlf_graph_node * len(graph))()
    for i, nd in enumerate(graph):
        x = arr[i]
        x.op = OPS.get(nd["op"], DLF_OP_OTHER)
        ins = list(nd["inputs"])
        if len(ins) > 2:
            raise ValueError(f"node {i}: at most two inputs")
        x.n_inputs = len(ins)
        for j, v in enumerate(ins):
            x.inputs[j] = v
        x.dtype = DTYPES.get(nd["dtype"], nd["dtype"])
        x.flags = (DLF_NODE_OUTPUT if nd.get("output") else 0) | (DLF_NODE_TRAINING if nd.get("training") else 0)
        shp = tuple(nd["shape"])
        if len(shp) > 4:
            raise ValueError(f"node {i}: rank above 4")
        x.rank = len(shp)
        for d, v in enumerate(shp):
            x.shape[d] = v
        x.flops = int(nd.get("flops", 0))
    return arr


def dlf_fusion_plan(graph, ridge, overhead_frac):
    """Groups chosen by the library's fusion pass: a list of dicts with "nodes" (chain order),
    "saved" (bytes) and "net" (bytes), in order of their first node."""
    arr = graph_nodes(graph)
    count = ctypes.c_int32(0)
    cap = max(1, len(graph))        # groups are disjoint and hold two or more nodes each
    out = (dlf_fusion_group * cap)()
    _check(_lib.dlf_fusion_plan(arr, len(graph), float(ridge), float(overhead_frac), out, cap,
                                ctypes.byref(count)), "dlf_fusion_plan")
    return [{"nodes": list(out[i].nodes[:out[i].count]), "saved": int(out[i].saved_bytes),
             "net": float(out[i].net_benefit)} for i in range(count.value)]


def raw():
    """The ctypes library handle (for status-code tests that bypass the raising wrappers)."""
    return _lib
