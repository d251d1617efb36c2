"""Python binding of the h3attn C ABI (``include/h3attn.h``), via ctypes.

Argument marshalling only: every function here converts Python arguments
(torch tensors, nested span lists, streams) into the plain pointers and sizes
of the C call of the same name, calls it, and raises ``H3AttnError`` on a
non-OK status.  All computation happens in the library's CUDA kernels; there
is no fallback.  If the library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import sys
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_uint64, c_void_p

import numpy as np

from . import build as _build

H3ATTN_OK, H3ATTN_EINVAL, H3ATTN_EUNSUPPORTED, H3ATTN_ENOMEM, H3ATTN_ECUDA, H3ATTN_ETIMEOUT = range(6)
STATUS_NAMES = ["OK", "EINVAL", "EUNSUPPORTED", "ENOMEM", "ECUDA", "ETIMEOUT"]


class H3AttnError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{fn}: H3ATTN_{name}: {msg}")


class h3attn_span(ctypes.Structure):
    _fields_ = [("n_t", c_int32), ("n_h", c_int32), ("n_w", c_int32),
                ("start", c_double * 3), ("step", c_double * 3)]


class h3attn_doc(ctypes.Structure):
    _fields_ = [("spans", POINTER(h3attn_span)), ("n_spans", c_int32)]


class h3attn_plan_opts(ctypes.Structure):
    _fields_ = [("num_heads", c_int32), ("head_dim", c_int32), ("rope_dims", c_int32),
                ("rope_base", c_double)]


class h3attn_rope_opts(ctypes.Structure):
    _fields_ = [("rope_dims", c_int32), ("interleaved", c_int32), ("base", c_double), ("scaling", c_int32),
                ("factor", c_double), ("original_len", c_double), ("beta_fast", c_double), ("beta_slow", c_double),
                ("amplitude", c_double), ("n_axes", c_int32), ("axis", c_void_p)]


class h3attn_rope(ctypes.Structure):
    _fields_ = [("rope_dims", c_int32), ("interleaved", c_int32), ("n_axes", c_int32), ("amplitude", c_float),
                ("turns", c_uint64 * 64), ("axis", ctypes.c_uint8 * 64)]


class h3attn_cache(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("n_pages", c_int32), ("page_size", c_int32),
                ("num_kv_heads", c_int32), ("page_stride", c_int64), ("token_stride", c_int64), ("head_stride", c_int64)]


_SIGS = {
    "h3attn_plan_create": [POINTER(h3attn_doc), c_int32, POINTER(h3attn_plan_opts), c_void_p,
                           POINTER(c_void_p)],
    "h3attn_plan_destroy": [c_void_p],
    "h3attn_plan_info": [c_void_p, POINTER(c_int64), POINTER(c_int32), POINTER(c_int32),
                         POINTER(c_int32)],
    "h3attn_plan_copy_cu_seqlens": [c_void_p, c_void_p],
    "h3attn_plan_copy_positions": [c_void_p, c_void_p],
    "h3attn_plan_copy_rope_table": [c_void_p, c_void_p],
    "h3attn_qk_prologue": [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int64,
                           c_void_p, c_void_p, c_int64, c_float, c_void_p],
    "h3attn_forward": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64,
                       c_float, c_void_p, c_void_p],
    "h3attn_forward_fused_q": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64,
                               c_void_p, c_int64, c_float, c_float, c_void_p, c_void_p],
    "h3attn_fp8_quantize": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p,
                            c_void_p, c_void_p, c_void_p, c_void_p],
    "h3attn_plan_fp8_v_keys": [c_void_p, POINTER(c_int64)],
    "h3attn_plan_forward_kernels": [c_void_p, POINTER(c_int32)],
    "h3attn_qk_prologue_fp8": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int64,
                               c_float, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p],
    "h3attn_work_list_host": [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p,
                              POINTER(c_int64), POINTER(c_int32)],
    "h3attn_forward_fp8": [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                           c_int64, c_float, c_void_p, c_void_p],
    "h3attn_forward_noalloc": [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int64,
                               c_void_p, c_int64, c_float, c_void_p, c_void_p],
    "h3attn_plan_set_sparse": [c_void_p, c_int32, c_int32, c_void_p],
    "h3attn_plan_sparse_info": [c_void_p, POINTER(c_int32), POINTER(c_int32), POINTER(c_int32)],
    "h3attn_block_select": [c_void_p, c_void_p, c_void_p, c_int64, c_int32, c_int32, c_void_p, c_void_p, c_void_p],
    "h3attn_forward_sparse": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_int64,
                              c_float, c_void_p, c_void_p],
    "h3attn_plan_set_prefix": [c_void_p, c_int32, c_void_p],
    "h3attn_forward_prefix": [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p,
                              c_int64, c_float, c_void_p, c_void_p],
    "h3attn_walk_list_host": [c_int32, c_void_p, c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_int64,
                              c_void_p, c_void_p, c_int64, c_void_p, c_int64, POINTER(c_int64), POINTER(c_int32),
                              POINTER(c_int64), POINTER(c_int64), POINTER(c_int64)],
    "h3attn_plan_set_causal": [c_void_p, c_int32, c_void_p],
    "h3attn_forward_causal": [c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_float, c_void_p,
                              c_void_p],
    "h3attn_plan_set_tree": [c_void_p, c_int32, c_void_p],
    "h3attn_forward_tree": [c_void_p, c_void_p, c_int64, POINTER(h3attn_cache), c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                            c_int64, c_float, c_void_p, c_void_p],
    "h3attn_rope_init": [POINTER(h3attn_rope_opts), POINTER(h3attn_rope)],
    "h3attn_rotary": [POINTER(h3attn_rope), c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int32, c_void_p,
                      c_int64, c_void_p, c_int64, c_int32, c_int32, c_void_p],
    "h3attn_rotary_store": [POINTER(h3attn_rope), c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int32,
                            c_void_p, c_void_p, c_int64, POINTER(h3attn_cache), c_void_p, c_void_p],
    "h3attn_cache_move": [POINTER(h3attn_cache), c_void_p, c_void_p, c_int64, c_int32, c_void_p],
    "h3attn_get_device_error": [c_void_p, c_void_p],
    "h3attn_selftest_bounded_wait": [c_uint64, c_void_p],
    "h3attn_selftest_plan_wait": [c_void_p, c_uint64, c_void_p],
    "h3attn_selftest_tree_join": [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p],
}

_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Loads libh3attn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with packed_varlen_non_gb300.build.build()")
        lib = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = c_int32
        lib.h3attn_last_error.argtypes = []
        lib.h3attn_last_error.restype = c_char_p
        _lib = lib
    return _lib


def h3attn_last_error() -> str:
    return load().h3attn_last_error().decode()


def _check(status: int, fn: str):
    if status != H3ATTN_OK:
        raise H3AttnError(status, fn, h3attn_last_error())


def _torch():
    return sys.modules["torch"]  # (whoever passes tensors has it)


def _stream(stream, device=None) -> int | None:
    """The stream's handle; for None the current one of `device` (None: of the
    current device)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


# The device that was current when a plan was created.
_plan_device: dict = {}


def _plan_stream(plan, stream):
    return _stream(stream, _plan_device.get(plan))


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _row_stride(t, given):
    if given is not None:
        return int(given)
    if isinstance(t, int):
        raise ValueError("a row stride is required when passing raw pointers")
    return int(t.stride(0))


# ------------------------------------------------------------------ plan ----

def h3attn_plan_create(docs, num_heads: int, rope_base: float = 10000.0, head_dim: int = 128,
                       rope_dims: int = 96, stream=None) -> int:
    """docs: list of documents, each a list of spans (n_t, n_h, n_w, start3, step3).
    Returns the opaque plan handle (an int)."""
    span_arrays = []
    cdocs = (h3attn_doc * max(1, len(docs)))()
    for i, d in enumerate(docs):
        arr = (h3attn_span * max(1, len(d)))()
        for j, (n_t, n_h, n_w, start, step) in enumerate(d):
            arr[j].n_t, arr[j].n_h, arr[j].n_w = int(n_t), int(n_h), int(n_w)
            for a in range(3):
                arr[j].start[a] = float(start[a])
                arr[j].step[a] = float(step[a])
        span_arrays.append(arr)
        cdocs[i].spans = ctypes.cast(arr, POINTER(h3attn_span))
        cdocs[i].n_spans = len(d)
    opts = h3attn_plan_opts(int(num_heads), int(head_dim), int(rope_dims), float(rope_base))
    out = c_void_p()
    st = _stream(stream) if stream is not False else None
    _check(load().h3attn_plan_create(cdocs, len(docs), ctypes.byref(opts), st, ctypes.byref(out)),
           "h3attn_plan_create")
    if "torch" in sys.modules:
        _plan_device[out.value] = _torch().cuda.current_device()
    return out.value


def h3attn_plan_destroy(plan):
    for known in (_list_sizes, _plan_rows, _prefix_rows, _causal_heads, _tree_docs, _plan_device):
        known.pop(plan, None)
    _check(load().h3attn_plan_destroy(plan), "h3attn_plan_destroy")


def h3attn_plan_info(plan) -> dict:
    S, nd, ml, nh = c_int64(), c_int32(), c_int32(), c_int32()
    _check(load().h3attn_plan_info(plan, ctypes.byref(S), ctypes.byref(nd), ctypes.byref(ml),
                                   ctypes.byref(nh)), "h3attn_plan_info")
    return {"S": S.value, "n_docs": nd.value, "max_seqlen": ml.value, "num_heads": nh.value}


def h3attn_plan_copy_cu_seqlens(plan) -> np.ndarray:
    info = h3attn_plan_info(plan)
    out = np.zeros(info["n_docs"] + 1, dtype=np.int32)
    _check(load().h3attn_plan_copy_cu_seqlens(plan, out.ctypes.data), "h3attn_plan_copy_cu_seqlens")
    return out


def h3attn_plan_copy_positions(plan) -> np.ndarray:
    info = h3attn_plan_info(plan)
    out = np.zeros((info["S"], 3), dtype=np.float64)
    _check(load().h3attn_plan_copy_positions(plan, out.ctypes.data), "h3attn_plan_copy_positions")
    return out


def h3attn_plan_copy_rope_table(plan) -> np.ndarray:
    info = h3attn_plan_info(plan)
    out = np.zeros((info["S"], 48, 2), dtype=np.float32)
    _check(load().h3attn_plan_copy_rope_table(plan, out.ctypes.data), "h3attn_plan_copy_rope_table")
    return out


# --------------------------------------------------------------- compute ----

def h3attn_qk_prologue(plan, q_in, k_in, q_out, k_out, gain_q, gain_k, eps: float = 1e-6,
                       in_row_stride=None, out_row_stride=None, gain_head_stride: int = 0,
                       stream=None):
    """Tensors: bf16 [S, H, 128]-shaped views (row stride taken from dim 0)
    or raw device pointers with explicit strides; gains fp32 on the device.
    q_in = q_out = None processes k only (for h3attn_forward_fused_q)."""
    for pair in ((q_in, k_in, in_row_stride), (q_out, k_out, out_row_stride)):
        if (pair[2] is None and pair[0] is not None and not isinstance(pair[0], int)
                and pair[0].stride(0) != pair[1].stride(0)):
            raise ValueError("q and k must share one row stride on each side")
    _check(load().h3attn_qk_prologue(plan, _ptr(q_in), _ptr(k_in), _row_stride(k_in, in_row_stride),
                                     _ptr(q_out), _ptr(k_out), _row_stride(k_out, out_row_stride),
                                     _ptr(gain_q), _ptr(gain_k), int(gain_head_stride), float(eps),
                                     _stream(stream)), "h3attn_qk_prologue")


def h3attn_forward(plan, q, k, v, o, softmax_scale: float, lse=None, qkv_row_stride=None,
                   o_row_stride=None, stream=None):
    if qkv_row_stride is None and not isinstance(q, int):
        strides = {int(x.stride(0)) for x in (q, k, v)}
        if len(strides) != 1:
            raise ValueError(f"q, k and v must share one row stride (got {sorted(strides)})")
    _check(load().h3attn_forward(plan, _ptr(q), _ptr(k), _ptr(v), _row_stride(q, qkv_row_stride),
                                 _ptr(o), _row_stride(o, o_row_stride), float(softmax_scale),
                                 _ptr(lse), _stream(stream)), "h3attn_forward")


def h3attn_forward_fused_q(plan, q_raw, k, v, o, gain_q, softmax_scale: float, eps: float = 1e-6,
                           lse=None, qkv_row_stride=None, o_row_stride=None, gain_head_stride: int = 0,
                           stream=None):
    """Forward with the Q prologue fused in: q_raw holds raw queries, k is
    already k-hat (see include/h3attn.h)."""
    if qkv_row_stride is None and not isinstance(q_raw, int):
        strides = {int(x.stride(0)) for x in (q_raw, k, v)}
        if len(strides) != 1:
            raise ValueError(f"q, k and v must share one row stride (got {sorted(strides)})")
    _check(load().h3attn_forward_fused_q(plan, _ptr(q_raw), _ptr(k), _ptr(v), _row_stride(q_raw, qkv_row_stride),
                                         _ptr(o), _row_stride(o, o_row_stride), _ptr(gain_q),
                                         int(gain_head_stride), float(eps), float(softmax_scale), _ptr(lse),
                                         _stream(stream)), "h3attn_forward_fused_q")


def h3attn_fp8_quantize(plan, q_hat, k_hat, v, q8, k8, v8t, sq, sk, sv, qkv_row_stride=None, stream=None):
    """FP8 quantisation of q-hat, k-hat, v (see include/h3attn.h for layouts)."""
    if qkv_row_stride is None and not isinstance(q_hat, int):
        strides = {int(x.stride(0)) for x in (q_hat, k_hat, v)}
        if len(strides) != 1:
            raise ValueError(f"q, k and v must share one row stride (got {sorted(strides)})")
    _check(load().h3attn_fp8_quantize(plan, _ptr(q_hat), _ptr(k_hat), _ptr(v), _row_stride(q_hat, qkv_row_stride),
                                      _ptr(q8), _ptr(k8), _ptr(v8t), _ptr(sq), _ptr(sk), _ptr(sv), _stream(stream)),
           "h3attn_fp8_quantize")


def h3attn_qk_prologue_fp8(plan, q_in, k_in, v, gain_q, gain_k, eps: float, q8, k8, v8t, sq, sk, sv,
                           gain_head_stride: int = 0, qkv_row_stride=None, stream=None):
    """The q/k prologue fused with the FP8 quantisation (see include/h3attn.h)."""
    if qkv_row_stride is None and not isinstance(q_in, int):
        strides = {int(x.stride(0)) for x in (q_in, k_in, v)}
        if len(strides) != 1:
            raise ValueError(f"q, k and v must share one row stride (got {sorted(strides)})")
    _check(load().h3attn_qk_prologue_fp8(plan, _ptr(q_in), _ptr(k_in), _ptr(v), _row_stride(q_in, qkv_row_stride),
                                         _ptr(gain_q), _ptr(gain_k), int(gain_head_stride), float(eps), _ptr(q8),
                                         _ptr(k8), _ptr(v8t), _ptr(sq), _ptr(sk), _ptr(sv), _stream(stream)),
           "h3attn_qk_prologue_fp8")


def h3attn_plan_forward_kernels(plan) -> int:
    n = c_int32()
    _check(load().h3attn_plan_forward_kernels(plan, ctypes.byref(n)), "h3attn_plan_forward_kernels")
    return n.value


def h3attn_work_list_host(cu_seqlens, num_heads: int, n_pairs: int):
    """The forward's work list for a layout, built on the host (no GPU needed).
    Returns (units int32 [n, 8], unit_off int32 [pairs + 1]); the fields of a
    unit are those of the C call."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    n_docs = int(cu.size) - 1
    n, used = c_int64(), c_int32()
    lib = load()
    _check(lib.h3attn_work_list_host(cu.ctypes.data, n_docs, int(num_heads), int(n_pairs), None, 0, None,
                                     ctypes.byref(n), ctypes.byref(used)), "h3attn_work_list_host")
    units = np.zeros((n.value, 8), dtype=np.int32)
    off = np.zeros(used.value + 1, dtype=np.int32)
    _check(lib.h3attn_work_list_host(cu.ctypes.data, n_docs, int(num_heads), int(n_pairs), units.ctypes.data,
                                     n.value, off.ctypes.data, ctypes.byref(n), ctypes.byref(used)),
           "h3attn_work_list_host")
    return units, off


def h3attn_plan_fp8_v_keys(plan) -> int:
    n = c_int64()
    _check(load().h3attn_plan_fp8_v_keys(plan, ctypes.byref(n)), "h3attn_plan_fp8_v_keys")
    return n.value


def h3attn_forward_fp8(plan, q8, k8, v8t, sq, sk, sv, o, softmax_scale: float, lse=None, o_row_stride=None,
                       stream=None):
    _check(load().h3attn_forward_fp8(plan, _ptr(q8), _ptr(k8), _ptr(v8t), _ptr(sq), _ptr(sk), _ptr(sv), _ptr(o),
                                     _row_stride(o, o_row_stride), float(softmax_scale), _ptr(lse),
                                     _stream(stream)), "h3attn_forward_fp8")


def h3attn_forward_noalloc(cu_seqlens, num_heads: int, q, k, v, o, softmax_scale: float, lse=None,
                           qkv_row_stride=None, o_row_stride=None, stream=None):
    """The allocation-free forward: cu_seqlens is a host int32 sequence
    [n_docs + 1]; no plan and no device allocation (see include/h3attn.h)."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    if qkv_row_stride is None and not isinstance(q, int):
        strides = {int(x.stride(0)) for x in (q, k, v)}
        if len(strides) != 1:
            raise ValueError(f"q, k and v must share one row stride (got {sorted(strides)})")
    _check(load().h3attn_forward_noalloc(cu.ctypes.data, cu.size - 1, int(num_heads), _ptr(q), _ptr(k),
                                         _ptr(v), _row_stride(q, qkv_row_stride), _ptr(o),
                                         _row_stride(o, o_row_stride), float(softmax_scale), _ptr(lse),
                                         _stream(stream)), "h3attn_forward_noalloc")


# ------------------------------------------------- sparse, shared prefix ----

# What the tensors of the walks' calls must be, of the plans that have them (fixed
# once set): (tokens, heads * 128, device), the prefix's rows, the lists' elements.
_plan_rows: dict = {}
_prefix_rows: dict = {}
_list_sizes: dict = {}


def _known(plan):
    """Notes the sizes of a plan that has just got a list."""
    info = h3attn_plan_info(plan)
    _plan_rows[plan] = (info["S"], info["num_heads"] * 128, _plan_device.get(plan))


def _on(x, device):
    """Whether a tensor lies on the given device (None: on any GPU)."""
    at = x.get_device()
    return at >= 0 if device is None else at == device


def _rows(tensors, given, rows, sizes):
    """The row stride shared by bf16 tensors of at least `rows` rows of
    heads * 128 contiguous elements on the plan's device; raw pointers among them
    are the caller's, with the given stride."""
    if sizes is None:  # the call itself refuses a plan without lists
        return _row_stride(tensors[0], given)
    _, width, device = sizes
    bf16 = _torch().bfloat16
    stride, shape, step, fits = given, None, None, False
    for x in tensors:
        if x is None or isinstance(x, int):
            continue
        last, shape, last_step, step = shape, x.shape, step, x.stride()
        if shape != last or step != last_step:  # (most calls' tensors are alike)
            n = len(shape)
            if n == 2:
                fits = step[1] == 1 and shape[1] >= width
            else:
                fits = n == 3 and step[2] == 1 and (step[1] == shape[2] or shape[1] == 1) and shape[1] * shape[2] >= width
            fits = fits and shape[0] >= rows
        at = x.get_device()
        if not fits or x.dtype is not bf16 or at < 0 or (device is not None and at != device):
            raise ValueError(f"a bfloat16 tensor of at least {rows} rows of {width} contiguous elements on the plan's "
                             f"device is needed (got {tuple(shape)}, strides {tuple(step)}, {x.dtype}, {x.device})")
        if rows == 1:
            continue  # (one row has no stride)
        if stride is None:
            stride = step[0]
        elif step[0] != stride:
            raise ValueError(f"tensors of one call must share one row stride (got {stride}, {step[0]})")
    if stride is None:
        if any(isinstance(x, int) for x in tensors):
            raise ValueError("a row stride is required when passing raw pointers")
        stride = width
    return int(stride)


def _check_lse(lse, sizes):
    if lse is None or isinstance(lse, int) or sizes is None:
        return
    n = sizes[0] * (sizes[1] // 128)
    if lse.dtype is not _torch().float32 or lse.numel() != n or not lse.is_contiguous() or not _on(lse, sizes[2]):
        raise ValueError(f"lse must be a contiguous float32 tensor of {n} elements on the plan's device "
                         f"(got {tuple(lse.shape)}, {lse.dtype}, {lse.device})")


def _check_lists(plan, block_idx, block_cnt):
    """The lists are read (or written) by their plan's sizes, so tensors must
    be int32, contiguous and of those sizes; raw pointers are the caller's."""
    sizes = _list_sizes.get(plan)
    if sizes is None:
        return  # the call itself refuses a plan without lists
    device = _plan_rows[plan][2]
    for t, n in ((block_idx, sizes[0]), (block_cnt, sizes[1])):
        if t is None or isinstance(t, int):
            continue
        if t.numel() != n or t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous() or not _on(t, device):
            raise ValueError("block_idx and block_cnt must be contiguous int32 tensors on the plan's device of "
                             f"{sizes[0]} and {sizes[1]} elements (got {tuple(t.shape)}, {t.dtype}, {t.device})")


def h3attn_plan_set_sparse(plan, q_block: int, max_blocks: int, stream=None):
    """Adds the block-sparse work list to a plan (once per plan)."""
    _check(load().h3attn_plan_set_sparse(plan, int(q_block), int(max_blocks), _plan_stream(plan, stream)),
           "h3attn_plan_set_sparse")
    info = h3attn_plan_sparse_info(plan)
    rows = info["num_heads"] * info["n_q_blocks"]
    _known(plan)
    _list_sizes[plan] = (rows * info["max_blocks"], rows)


def h3attn_plan_sparse_info(plan) -> dict:
    qb, mb, nq, nh = c_int32(), c_int32(), c_int32(), c_int32()
    _check(load().h3attn_plan_sparse_info(plan, ctypes.byref(qb), ctypes.byref(mb), ctypes.byref(nq)),
           "h3attn_plan_sparse_info")
    _check(load().h3attn_plan_info(plan, None, None, None, ctypes.byref(nh)), "h3attn_plan_info")
    return {"q_block": qb.value, "max_blocks": mb.value, "n_q_blocks": nq.value, "num_heads": nh.value}


def h3attn_block_select(plan, q_hat, k_hat, keep: int, block_idx, block_cnt, keep_own: bool = True,
                        qkv_row_stride=None, stream=None):
    """Scores and keeps key tiles: block_idx int32 [H, n_q_blocks, max_blocks],
    block_cnt int32 [H, n_q_blocks] (see include/h3attn.h)."""
    sizes = _plan_rows.get(plan)
    stride = _rows((q_hat, k_hat), qkv_row_stride, sizes[0] if sizes else 0, sizes)
    _check_lists(plan, block_idx, block_cnt)
    _check(load().h3attn_block_select(plan, _ptr(q_hat), _ptr(k_hat), stride, int(keep), int(bool(keep_own)),
                                      _ptr(block_idx), _ptr(block_cnt), _plan_stream(plan, stream)),
           "h3attn_block_select")


def h3attn_forward_sparse(plan, q, k, v, block_idx, block_cnt, o, softmax_scale: float, lse=None,
                          qkv_row_stride=None, o_row_stride=None, stream=None):
    """The forward over the listed key tiles of each query block."""
    sizes = _plan_rows.get(plan)
    rows = sizes[0] if sizes else 0
    stride = _rows((q, k, v), qkv_row_stride, rows, sizes)
    o_stride = _rows((o,), o_row_stride, rows, sizes)
    _check_lse(lse, sizes)
    _check_lists(plan, block_idx, block_cnt)
    _check(load().h3attn_forward_sparse(plan, _ptr(q), _ptr(k), _ptr(v), stride, _ptr(block_idx), _ptr(block_cnt),
                                        _ptr(o), o_stride, float(softmax_scale), _ptr(lse),
                                        _plan_stream(plan, stream)), "h3attn_forward_sparse")


def h3attn_plan_set_prefix(plan, prefix_len: int, stream=None):
    """Adds the work list for a shared prefix of prefix_len rows to a plan
    (once per plan)."""
    _check(load().h3attn_plan_set_prefix(plan, int(prefix_len), _plan_stream(plan, stream)),
           "h3attn_plan_set_prefix")
    _known(plan)
    _prefix_rows[plan] = int(prefix_len)


def h3attn_forward_prefix(plan, q, k, v, k_prefix, v_prefix, o, softmax_scale: float, lse=None,
                          qkv_row_stride=None, prefix_row_stride=None, o_row_stride=None, stream=None):
    """The forward of a batch whose documents all attend to one prefix besides
    themselves; k_prefix and v_prefix are bf16 [prefix_len, H, 128]-shaped."""
    sizes, prefix_len = _plan_rows.get(plan), _prefix_rows.get(plan)
    rows = sizes[0] if sizes else 0
    stride = _rows((q, k, v), qkv_row_stride, rows, sizes)
    prefix_stride = _rows((k_prefix, v_prefix), prefix_row_stride, prefix_len, sizes if prefix_len else None)
    o_stride = _rows((o,), o_row_stride, rows, sizes)
    _check_lse(lse, sizes)
    _check(load().h3attn_forward_prefix(plan, _ptr(q), _ptr(k), _ptr(v), stride, _ptr(k_prefix), _ptr(v_prefix),
                                        prefix_stride, _ptr(o), o_stride, float(softmax_scale), _ptr(lse),
                                        _plan_stream(plan, stream)), "h3attn_forward_prefix")


def h3attn_walk_list_host(kind: int, cu_seqlens, num_heads: int, p0: int, p1: int, n_pairs: int):
    """The work list of the sparse (kind 0: p0 = q_block, p1 = max_blocks), prefix
    (kind 1: p0 = prefix_len) or causal (kind 2: p0 = num_kv_heads) forward, built on the host: (units [n, 8],
    unit_off, joins [m, 12], own tiles [t, 20], partial rows); the fields are
    those of the C call."""
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    n, used, nj, no, rows = c_int64(), c_int32(), c_int64(), c_int64(), c_int64()
    head = (int(kind), cu.ctypes.data, int(cu.size) - 1, int(num_heads), int(p0), int(p1), int(n_pairs))
    tail = [ctypes.byref(x) for x in (n, used, nj, no, rows)]
    lib = load()
    _check(lib.h3attn_walk_list_host(*head, None, 0, None, None, 0, None, 0, *tail), "h3attn_walk_list_host")
    units = np.zeros((n.value, 8), dtype=np.int32)
    off = np.zeros(used.value + 1, dtype=np.int32)
    joins = np.zeros((nj.value, 12), dtype=np.int32)
    own = np.zeros((no.value, 20), dtype=np.int32)
    _check(lib.h3attn_walk_list_host(*head, units.ctypes.data, n.value, off.ctypes.data, joins.ctypes.data, nj.value,
                                     own.ctypes.data, no.value, *tail), "h3attn_walk_list_host")
    return units, off, joins, own, rows.value


# ------------------------------------------------------ causal, grouped ----

_causal_heads: dict = {}  # key heads of the plans that have a causal list


def h3attn_plan_set_causal(plan, num_kv_heads: int, stream=None):
    """Adds the causal work list to a plan (once per plan)."""
    _check(load().h3attn_plan_set_causal(plan, int(num_kv_heads), _plan_stream(plan, stream)), "h3attn_plan_set_causal")
    _known(plan)
    _causal_heads[plan] = int(num_kv_heads)


def h3attn_forward_causal(plan, q, k, v, o, softmax_scale: float, lse=None, q_row_stride=None, kv_row_stride=None,
                          o_row_stride=None, stream=None):
    """Causal attention over the plan's documents with grouped heads: q, o bf16 [S, H, 128]-shaped, k and v
    [S, num_kv_heads, 128]-shaped, each side with a row stride of its own."""
    sizes, kv = _plan_rows.get(plan), _causal_heads.get(plan)
    rows = sizes[0] if sizes else 0
    q_stride = _rows((q,), q_row_stride, rows, sizes)
    kv_stride = _rows((k, v), kv_row_stride, rows, (rows, 128 * kv, sizes[2]) if kv else None)
    o_stride = _rows((o,), o_row_stride, rows, sizes)
    _check_lse(lse, sizes)
    _check(load().h3attn_forward_causal(plan, _ptr(q), q_stride, _ptr(k), _ptr(v), kv_stride, _ptr(o), o_stride,
                                        float(softmax_scale), _ptr(lse), _plan_stream(plan, stream)), "h3attn_forward_causal")


# ------------------------------------------------ positions, paged cache ----

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def h3attn_rope_init(rope_dims: int = 128, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                     factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     amplitude: float = 0.0, axes=None, n_axes=None) -> h3attn_rope:
    """Frequencies of a rotary embedding (host data for the rotary calls); scaling is "none",
    "linear", "ntk" or "parts", axes the position axis of each of the rope_dims / 2 pairs."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)} (got {scaling!r})")
    axis = None
    if axes is not None:
        if len(axes) != int(rope_dims) // 2:
            raise ValueError(f"axes must name the axis of each of {int(rope_dims) // 2} pairs (got {len(axes)})")
        if any(not 0 <= int(x) < 3 for x in axes):
            raise ValueError("axes must be 0, 1 or 2")
        axis = np.asarray([int(x) for x in axes], dtype=np.uint8)
        n_axes = int(axis.max()) + 1 if n_axes is None and axis.size else n_axes
    opts = h3attn_rope_opts(int(rope_dims), int(bool(interleaved)), float(base), _SCALINGS[scaling], float(factor),
                            float(original_len), float(beta_fast), float(beta_slow), float(amplitude), int(n_axes or 1),
                            axis.ctypes.data if axis is not None else None)
    out = h3attn_rope()
    _check(load().h3attn_rope_init(ctypes.byref(opts), ctypes.byref(out)), "h3attn_rope_init")
    return out


class Cache:
    """The caller's cache: bf16 tensors k and v of [pages, tokens of a page, heads, 128], of any
    strides but the last (a head-major one is a transposed view)."""

    def __init__(self, k, v):
        for x in (k, v):
            if (x.dtype is not _torch().bfloat16 or x.dim() != 4 or x.shape[3] != 128 or x.stride(3) != 1
                    or x.get_device() < 0 or x.shape != k.shape or x.stride() != k.stride() or x.device != k.device):
                raise ValueError("a cache is two bfloat16 tensors [pages, tokens, heads, 128] on one GPU with equal strides "
                                 f"and a contiguous last dimension (got {tuple(x.shape)}, strides {x.stride()}, "
                                 f"{x.dtype}, {x.device})")
        self.k, self.v, self.device = k, v, k.get_device()
        self.num_kv_heads = k.shape[2]
        self.c = h3attn_cache(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[1], k.shape[2], k.stride(0), k.stride(1),
                              k.stride(2))


def _bad_rows(x, name, n, device):
    return ValueError(f"{name} must be a bfloat16 tensor [{n}, heads, 128] with contiguous heads on GPU {device} "
                      f"(got {tuple(x.shape)}, strides {x.stride()}, {x.dtype}, {x.device})")


def _heads(x, name, n, device, bf16):
    """(pointer, row stride, heads) of bf16 rows [n, heads, 128] on the device."""
    if x.dtype is bf16 and x.dim() == 3 and x.get_device() == device >= 0:
        rows, heads, dims = x.shape
        step, head, dim = x.stride()
        if rows == n and dims == 128 and dim == 1 and (head == 128 or heads == 1):
            return x.data_ptr(), (step if n > 1 else 128 * heads), heads
    raise _bad_rows(x, name, n, device)


def _ints(x, name, shape, device):
    """The pointer of a contiguous int32 tensor of the given shape on the device."""
    if x.shape != shape or x.dtype is not _torch().int32 or x.get_device() != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on GPU {device} "
                         f"(got {tuple(x.shape)}, {x.dtype}, {x.device})")
    return x.data_ptr()


def _positions(rope, positions, n, device):
    axes = rope.n_axes
    return _ints(positions, "positions", (n,) if axes == 1 and positions.dim() == 1 else (axes, n), device)


_NO_ROWS = (None, 0, 0)


def _call_on(device, fn, name, stream, *args):
    """The call without a plan, with the tensors' device current."""
    c = _torch()._C
    at = c._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if c._cuda_getDevice() == device:
        status = fn(*args, at)
    else:
        with _torch().cuda.device(device):
            status = fn(*args, at)
    if status != H3ATTN_OK:
        _check(status, name)


def h3attn_rotary(rope, positions, q_in, q_out, k_in=None, k_out=None, inverse: bool = False, stream=None):
    """Rotates q (and k): bf16 tensors [n, heads, 128], each with a row stride of its own; positions
    int32 [n_axes, n] ([n] for one axis).  q_in and q_out, or k_in and k_out, may both be None."""
    first = q_in if q_in is not None else k_in
    if first is None or (q_in is None) != (q_out is None) or (k_in is None) != (k_out is None):
        raise ValueError("an input and its output go together, and one pair is needed")
    n, device, bf16 = first.shape[0], first.get_device(), _torch().bfloat16
    q, q_step, heads = q2, q2_step, heads2 = k, k_step, kv = k2, k2_step, kv2 = _NO_ROWS
    if q_in is not None:
        q, q_step, heads = _heads(q_in, "q_in", n, device, bf16)
        q2, q2_step, heads2 = _heads(q_out, "q_out", n, device, bf16)
    if k_in is not None:
        k, k_step, kv = _heads(k_in, "k_in", n, device, bf16)
        k2, k2_step, kv2 = _heads(k_out, "k_out", n, device, bf16)
    if heads != heads2 or kv != kv2:
        raise ValueError("an input and its output must have the same heads")
    _call_on(device, load().h3attn_rotary, "h3attn_rotary", stream, rope, _positions(rope, positions, n, device), n, q, q_step, q2,
             q2_step, heads, k, k_step, k2, k2_step, kv, 1 if inverse else 0)


def h3attn_rotary_store(rope, positions, q_in, q_out, k_in, v_in, cache: Cache, slots, stream=None):
    """Rotates q into q_out (both may be None) and k into the cache, and copies v beside it; slots
    int32 [n]."""
    if (q_in is None) != (q_out is None):
        raise ValueError("q_in and q_out go together")
    n, device, bf16 = k_in.shape[0], cache.device, _torch().bfloat16
    q, q_step, heads = q2, q2_step, heads2 = _NO_ROWS
    if q_in is not None:
        q, q_step, heads = _heads(q_in, "q_in", n, device, bf16)
        q2, q2_step, heads2 = _heads(q_out, "q_out", n, device, bf16)
    k, k_step, kv = _heads(k_in, "k_in", n, device, bf16)
    v, v_step, kv2 = _heads(v_in, "v_in", n, device, bf16)
    if heads != heads2 or kv != cache.num_kv_heads or kv2 != kv:
        raise ValueError("q_in and q_out must have the same heads, and k_in and v_in the cache's")
    if k_step != v_step:
        raise ValueError(f"k_in and v_in must share one row stride (got {k_step}, {v_step})")
    _call_on(device, load().h3attn_rotary_store, "h3attn_rotary_store", stream, rope, _positions(rope, positions, n, device), n, q,
             q_step, q2, q2_step, heads, k, v, k_step, cache.c, _ints(slots, "slots", (n,), device))


def h3attn_cache_move(cache: Cache, src, dst, stream=None):
    """Copies rows of the cache to other slots: src, dst int32 [groups, width]."""
    if src.dim() != 2:
        raise ValueError(f"src and dst are [groups, width] (got {tuple(src.shape)})")
    shape = src.shape
    _call_on(cache.device, load().h3attn_cache_move, "h3attn_cache_move", stream, cache.c, _ints(src, "src", shape, cache.device),
             _ints(dst, "dst", shape, cache.device), shape[0], shape[1])


_tree_docs: dict = {}  # documents of the plans that have a tree workspace


def h3attn_plan_set_tree(plan, num_kv_heads: int, stream=None):
    """Adds the tree forward's workspace to a plan whose documents are trees of drafts (once per plan)."""
    _check(load().h3attn_plan_set_tree(plan, int(num_kv_heads), _plan_stream(plan, stream)), "h3attn_plan_set_tree")
    _known(plan)
    _tree_docs[plan] = h3attn_plan_info(plan)["n_docs"]


def h3attn_forward_tree(plan, q, cache: Cache, page_table, ctx_lens, o, softmax_scale: float, lse=None, tree_mask=None,
                        q_row_stride=None, o_row_stride=None, stream=None):
    """Attention of drafted tokens over their sequences' pages: q, o bf16 [S, H, 128]-shaped, page_table int32
    [n_docs, width], ctx_lens int32 [n_docs], tree_mask int64 or uint64 [S] (None: each draft sees those before it)."""
    sizes, docs = _plan_rows.get(plan), _tree_docs.get(plan)
    rows = sizes[0] if sizes else 0
    q_stride = _rows((q,), q_row_stride, rows, sizes)
    o_stride = _rows((o,), o_row_stride, rows, sizes)
    _check_lse(lse, sizes)
    if docs is None:  # the call itself refuses a plan without a workspace
        width, table, ctx = 1, 0, 0
    else:
        if page_table.dim() != 2:
            raise ValueError(f"page_table is [n_docs, width] (got {tuple(page_table.shape)})")
        width = page_table.shape[1]
        table = _ints(page_table, "page_table", (docs, width), cache.device)
        ctx = _ints(ctx_lens, "ctx_lens", (docs,), cache.device)
        if sizes[2] is not None and cache.device != sizes[2]:
            raise ValueError(f"the cache lies on GPU {cache.device}, the plan on {sizes[2]}")
        if tree_mask is not None and not isinstance(tree_mask, int) and (
                tree_mask.dtype not in (_torch().int64, _torch().uint64) or not tree_mask.is_contiguous()
                or tuple(tree_mask.shape) != (rows,) or tree_mask.get_device() != cache.device):
            raise ValueError(f"tree_mask must be a contiguous int64 or uint64 tensor ({rows},) on GPU {cache.device} "
                             f"(got {tuple(tree_mask.shape)}, {tree_mask.dtype}, {tree_mask.device})")
    _check(load().h3attn_forward_tree(plan, _ptr(q), q_stride, cache.c, table, width, ctx, _ptr(tree_mask), _ptr(o), o_stride,
                                      float(softmax_scale), _ptr(lse), _plan_stream(plan, stream)), "h3attn_forward_tree")


def h3attn_get_device_error(plan, stream=None):
    _check(load().h3attn_get_device_error(plan, _plan_stream(plan, stream)), "h3attn_get_device_error")


def h3attn_selftest_bounded_wait(timeout_ns: int, stream=None) -> int:
    """Returns the raw status (ETIMEOUT is the expected outcome)."""
    return int(load().h3attn_selftest_bounded_wait(int(timeout_ns), _stream(stream)))


def h3attn_selftest_plan_wait(plan, timeout_ns: int, stream=None):
    """A wait that runs out, recorded in the plan's device error word."""
    _check(load().h3attn_selftest_plan_wait(plan, int(timeout_ns), _plan_stream(plan, stream)), "h3attn_selftest_plan_wait")


def h3attn_selftest_tree_join(plan, o, lse=None, joins=None, o_row_stride=None, stream=None):
    """The tree forward's join by itself, on the plan's entries or on joins (int32 [items, 2])."""
    sizes = _plan_rows.get(plan)
    stride = _rows((o,), o_row_stride, sizes[0] if sizes else 0, sizes)
    _check_lse(lse, sizes)
    n = 0
    if joins is not None:
        n = joins.shape[0]
        _ints(joins, "joins", (n, 2), o.get_device())
    _check(load().h3attn_selftest_tree_join(plan, _ptr(joins), n, _ptr(o), stride, _ptr(lse), _plan_stream(plan, stream)),
           "h3attn_selftest_tree_join")


class Plan:
    """Owns a plan handle; a context manager around create/destroy."""

    def __init__(self, docs, num_heads, rope_base=10000.0, stream=None):
        self.handle = h3attn_plan_create(docs, num_heads, rope_base, stream=stream)
        self.info = h3attn_plan_info(self.handle)

    def close(self):
        if self.handle:
            h3attn_plan_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
