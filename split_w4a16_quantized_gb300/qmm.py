"""Python binding of libqmm (ctypes): argument marshalling only.

Every function here has the name of the C entry point it calls (include/qmm.h)
and hands device pointers, sizes and the current CUDA stream to it; all
arithmetic runs in the library's CUDA kernels.  torch is used for device
memory and streams only.  If libqmm.so has not been built the first call
raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

QMM_OK, QMM_EINVAL, QMM_ESHAPE, QMM_EWORKSPACE, QMM_ECUDA, QMM_EALIGN, QMM_ENODEV = \
    0, -1, -2, -3, -4, -5, -6

QMM_PARTIAL_BF16, QMM_PARTIAL_F32 = 0, 1
QMM_PRESET_PAGES, QMM_PRESET_GB300 = 0, 1
QMM_KERNELS_DEFAULT, QMM_KERNELS_MMA_SYNC, QMM_KERNELS_TCGEN05, QMM_KERNELS_LEAN = 0, 1, 2, 3


class qmm_policy(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int), ("bn", ctypes.c_int), ("target_blocks", ctypes.c_int),
                ("cap", ctypes.c_int), ("min_k_per_split", ctypes.c_int)]

    def as_tuple(self):
        return (self.bm, self.bn, self.target_blocks, self.cap, self.min_k_per_split)

    def __repr__(self):
        return "qmm_policy(bm=%d, bn=%d, target_blocks=%d, cap=%d, min_k_per_split=%d)" % \
            self.as_tuple()


QMM_OPT_DEFAULT = -1
_OPTION_FIELDS = ("kernels", "partitions", "reduce", "weights_static", "pdl",
                  "grouped_schedule", "group_plan")


class qmm_options(ctypes.Structure):
    """Per-call options (see qmm.h); every field defaults to QMM_OPT_DEFAULT."""
    _fields_ = [(f, ctypes.c_int) for f in _OPTION_FIELDS]

    def __init__(self, **kw):
        super().__init__(*([QMM_OPT_DEFAULT] * len(_OPTION_FIELDS)))
        for k, v in kw.items():
            if k not in _OPTION_FIELDS:
                raise TypeError("unknown option %r" % k)
            setattr(self, k, int(v))


def _opt(options):
    return ctypes.byref(options) if options is not None else None


class QmmError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = " [%s]" % qmm_last_cuda_error() if code == QMM_ECUDA else ""
        super().__init__("%s: %s (%d)%s" % (what, qmm_strerror(code), code, detail))


class qmm_stream_call(ctypes.Structure):
    """One chunk of qmm_w4a16_g128_stream (see qmm.h)."""
    _fields_ = [("A_host", ctypes.c_void_p), ("C_host", ctypes.c_void_p),
                ("Wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("M", ctypes.c_int), ("Kred", ctypes.c_int),
                ("Nout", ctypes.c_int)]


class qmm_group_call(ctypes.Structure):
    """One call of qmm_w4a16_g128_grouped (see qmm.h)."""
    _fields_ = [("A", ctypes.c_void_p), ("Wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("C", ctypes.c_void_p), ("M", ctypes.c_int),
                ("Kred", ctypes.c_int), ("Nout", ctypes.c_int)]


class qmm_kv_cache(ctypes.Structure):
    """The paged KV cache of one layer (see qmm.h); kv_cache() builds it."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("B", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class qmm_rope(ctypes.Structure):
    """Rotation and per-head norm of qmm_kv_append (see qmm.h); rope() builds it."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("rows", ctypes.c_int), ("dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("eps", ctypes.c_float)]


class qmm_rope_axes(ctypes.Structure):
    """Axis of each rotated pair of qmm_kv_append_axes (see qmm.h); rope_axes() builds it."""
    _fields_ = [("axes", ctypes.c_int), ("axis", ctypes.c_uint8 * 64)]


class qmm_prefix(ctypes.Structure):
    """Prefixes shared by runs of sequences (see qmm.h); prefix() builds it."""
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("G", ctypes.c_int), ("max_pages", ctypes.c_int)]


_lock = threading.Lock()
_lib = None

_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L = ctypes.c_int64
_SIGS = {
    "qmm_policy_preset": (_I, [_I, _I, _I, ctypes.POINTER(qmm_policy)]),
    "qmm_kernel_tile": (_I, [_I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "qmm_kernel_grouped": (_I, [_I]),
    "qmm_splitk_plan": (_I, [_I, _I, _I, ctypes.POINTER(qmm_policy), ctypes.POINTER(_I)]),
    "qmm_splitk_plan_near_equal": (_I, [_I, _I, _I, ctypes.POINTER(qmm_policy),
                                        ctypes.POINTER(_I)]),
    "qmm_splitk_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "qmm_w4a16_g128": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(qmm_policy),
                            _P, _SZ, _I, _P, ctypes.POINTER(_I)]),
    "qmm_splitk_reduce": (_I, [_P, _I, _I, _I, _I, _P, _P]),
    "qmm_w4a16_g128_partition": (_I, [_P, _P, _P, _P, _P, _SZ, _I, _I, _I, _I, _I, _P]),
    "qmm_gemm_bf16_splitk": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qmm_gemm_workspace_bytes": (_SZ, [_I, _I, _I]),
    "qmm_unpack_probe": (_I, [_P, _I, _I, _P, _P]),
    "qmm_dequant_probe": (_I, [_P, _P, _P, _I, _I, _P, _P]),
    "qmm_strerror": (ctypes.c_char_p, [_I]),
    "qmm_last_cuda_error": (ctypes.c_char_p, []),
    "qmm_options_init": (None, [_P]),
    "qmm_w4a16_g128_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(qmm_policy),
                               _P, _SZ, _I, _P, ctypes.POINTER(_I), _P]),
    "qmm_splitk_workspace_bytes_ex": (_SZ, [_I, _I, _I, _I, _P]),
    "qmm_call_plan": (_I, [_I, _I, _I, _I, ctypes.POINTER(qmm_policy), _I, _I, _P,
                           ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I),
                           ctypes.POINTER(_I)]),
    "qmm_call_workspace_bytes": (_SZ, [_I, _I, _I, _I, ctypes.POINTER(qmm_policy), _I, _I, _P]),
    "qmm_set_kernels": (_I, [_I]),
    "qmm_set_pdl": (_I, [_I]),
    "qmm_set_weights_static": (_I, [_I]),
    "qmm_set_reduce": (_I, [_I]),
    "qmm_set_partitions": (_I, [_I]),
    "qmm_set_grouped_schedule": (_I, [_I]),
    "qmm_set_group_plan": (_I, [_I]),
    "qmm_group_plan": (_I, [ctypes.POINTER(_I), _I, _I, _I, ctypes.POINTER(_I)]),
    "qmm_kernel_status": (_I, [ctypes.POINTER(_I), _I]),
    "qmm_wait_timeout_probe": (_I, [ctypes.c_void_p]),
    "qmm_w4a16_g128_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I,
                                    ctypes.POINTER(qmm_policy), _I, _P, ctypes.POINTER(_I)]),
    "qmm_static_scratch_bytes": (_SZ, []),
    "qmm_tc_pipeline_config": (_I, [_I, _I, _I, ctypes.POINTER(_I)]),
    "qmm_tc_persistent_pipeline_config": (_I, [_I, _I, _I, ctypes.POINTER(_I)]),
    "qmm_decode_attention_splits": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "qmm_decode_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "qmm_decode_attention": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _I,
                                  _P, _SZ, _P, ctypes.POINTER(_I)]),
    "qmm_group_workspace_bytes": (_SZ, [ctypes.POINTER(qmm_group_call), _I, _I]),
    "qmm_w4a16_g128_grouped": (_I, [ctypes.POINTER(qmm_group_call), _I, _P, _SZ, _I, _P,
                                    ctypes.POINTER(_I)]),
    "qmm_group_workspace_bytes_ex": (_SZ, [ctypes.POINTER(qmm_group_call), _I, _I, _P]),
    "qmm_w4a16_g128_grouped_ex": (_I, [ctypes.POINTER(qmm_group_call), _I, _P, _SZ, _I, _P,
                                       ctypes.POINTER(_I), _P]),
    "qmm_stream_arena_bytes": (_SZ, [ctypes.POINTER(qmm_stream_call), _I, _I]),
    "qmm_w4a16_g128_stream": (_I, [ctypes.POINTER(qmm_stream_call), _I, _I, _P, _SZ, _P, _P, _P,
                                   ctypes.POINTER(_I)]),
    "qmm_kv_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _L, _L, _L, _L, _P, _P, _P, _P]),
    "qmm_tree_attention": (_I, [_P, _P, _L, _P, _I, _I, _I, _P, _P, ctypes.c_float, _P, _SZ, _P]),
    "qmm_tree_attention_workspace_bytes": (_SZ, [_P, _I, _I, _I]),
    "qmm_kv_append_axes": (_I, [_P, _P, _P, _P, _P, _I, _I, _L, _L, _L, _L, _P, _P, _P, _P, _P]),
    "qmm_kv_evict": (_I, [_P, _I, _P, _P, _L, _L, _I, _I, _I, _P, _P, _P]),
    "qmm_prefix_attention": (_I, [_P, _P, _P, _L, _P, _I, _I, _I, _P, _P, ctypes.c_float, _P,
                                  _SZ, _P]),
    "qmm_prefix_attention_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I]),
    "qmm_scored_attention": (_I, [_P, _P, _L, _P, _I, _I, _I, _P, ctypes.c_float, _P, _L,
                                  ctypes.c_float, _P, _SZ, _P]),
    "qmm_scored_attention_workspace_bytes": (_SZ, [_P, _I, _I, _I]),
    "qmm_tree_accept": (_I, [_P, _I, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P]),
    "qmm_overlap_schedule": (_I, [_I, _I, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                  _I, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_double)]),
}


def lib() -> ctypes.CDLL:
    """The loaded libqmm.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libqmm.so is not built; run "
                                   "`python -m split_w4a16_quantized_gb300.build`")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _lib = h
        return _lib


def _check(rc: int, what: str):
    if rc != QMM_OK:
        raise QmmError(rc, what)


# torch's raw current-stream lookup: a plain integer, without building a
# torch.cuda.Stream object (about 3 µs of host time per call on an Arm host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _cur_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_cur_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtypes, name: str) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _ptr(t: torch.Tensor, dtypes, name: str) -> int:
    """_dev's checks in one expression for the per-call entry points; the
    pointer as a plain integer.  Any failed check is reported by _dev."""
    try:
        if t.is_cuda and t.dtype in dtypes and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtypes, name)
    raise TypeError("%s is not a usable CUDA tensor" % name)


_BF16 = (torch.bfloat16,)
_WORDS = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)


# ---- host-only entry points ---------------------------------------------

def qmm_strerror(code: int) -> str:
    return lib().qmm_strerror(code).decode()


def qmm_last_cuda_error() -> str:
    """Name of the CUDA error behind this thread's latest QMM_ECUDA."""
    return lib().qmm_last_cuda_error().decode()


def qmm_policy_preset(which: int, M: int = 1, num_sms: int = 0) -> qmm_policy:
    out = qmm_policy()
    _check(lib().qmm_policy_preset(which, M, num_sms, ctypes.byref(out)), "qmm_policy_preset")
    return out


def qmm_set_kernels(which: int) -> int:
    """Select the kernel table (QMM_KERNELS_*); returns the previous one."""
    prev = lib().qmm_set_kernels(which)
    if prev < 0:
        raise QmmError(prev, "qmm_set_kernels")
    return prev


def qmm_set_pdl(enable: bool) -> int:
    """Programmatic dependent launch on/off; returns the previous setting."""
    return lib().qmm_set_pdl(int(bool(enable)))


QMM_REDUCE_KERNEL, QMM_REDUCE_FUSED, QMM_REDUCE_CLUSTER = 0, 1, 2


def qmm_set_reduce(mode: int) -> int:
    """Separate reduce kernel (default), the fused last-CTA reduce or the
    cluster reduce (see qmm.h)."""
    prev = lib().qmm_set_reduce(mode)
    if prev < 0:
        raise QmmError(prev, "qmm_set_reduce")
    return prev


QMM_PARTITIONS_EQUAL, QMM_PARTITIONS_NEAR_EQUAL = 0, 1


def qmm_set_partitions(mode: int) -> int:
    """Equal partitions (default) or near-equal ones for any split (see qmm.h)."""
    prev = lib().qmm_set_partitions(mode)
    if prev < 0:
        raise QmmError(prev, "qmm_set_partitions")
    return prev


QMM_GROUPED_TILES, QMM_GROUPED_PERSISTENT = 0, 1


def qmm_set_grouped_schedule(mode: int) -> int:
    """Schedule of the grouped call's tcgen05 launches (QMM_GROUPED_*, the
    persistent one by default); returns the previous one."""
    prev = lib().qmm_set_grouped_schedule(mode)
    if prev < 0:
        raise QmmError(prev, "qmm_set_grouped_schedule")
    return prev


QMM_GROUP_PLAN_CALLS, QMM_GROUP_PLAN_GROUP = 0, 1
QMM_SPLIT_PLANNED = -1  # split_req of qmm_w4a16_g128: the group plan for the call alone
QMM_SPLIT_BALANCED = -2  # split_req: whole waves unsplit, the partial wave's rows split


def qmm_set_group_plan(mode: int) -> int:
    """Split plan of the grouped call (QMM_GROUP_PLAN_*); returns the previous one."""
    prev = lib().qmm_set_group_plan(mode)
    if prev < 0:
        raise QmmError(prev, "qmm_set_group_plan")
    return prev


def qmm_group_plan(shapes, num_sms: int = 0, partial_dtype: int = QMM_PARTIAL_BF16) -> list:
    """The group plan's splits for shapes [(M, Kred, Nout), ...] (host only)."""
    n = len(shapes)
    flat = (_I * (3 * n))(*[int(v) for shp in shapes for v in shp])
    out = (_I * n)()
    _check(lib().qmm_group_plan(flat, n, num_sms, partial_dtype, out), "qmm_group_plan")
    return list(out)


def qmm_set_weights_static(enable: bool) -> int:
    """Promise that no earlier kernel on the stream writes the weights (see qmm.h)."""
    return int(lib().qmm_set_weights_static(1 if enable else 0))


def qmm_kernel_status(clear: bool = True) -> int:
    """0, or 1 if a bounded wait inside a tcgen05 kernel ran out (synchronizes)."""
    st = _I(0)
    _check(lib().qmm_kernel_status(ctypes.byref(st), int(clear)), "qmm_kernel_status")
    return st.value


def qmm_wait_timeout_probe(stream=None) -> None:
    """Launch one CTA whose bounded wait runs out (test hook; see qmm.h)."""
    _check(lib().qmm_wait_timeout_probe(_stream(stream)), "qmm_wait_timeout_probe")


def qmm_kernel_tile(M: int):
    bm, bn = _I(0), _I(0)
    _check(lib().qmm_kernel_tile(M, ctypes.byref(bm), ctypes.byref(bn)), "qmm_kernel_tile")
    return bm.value, bn.value


def qmm_kernel_grouped(M: int) -> bool:
    """True if the grouped call runs calls with M rows in shared launches."""
    rc = lib().qmm_kernel_grouped(M)
    if rc < 0:
        _check(rc, "qmm_kernel_grouped")
    return rc == 1


def qmm_splitk_plan(M: int, Kred: int, Nout: int, pol: qmm_policy) -> int:
    s = _I(0)
    _check(lib().qmm_splitk_plan(M, Kred, Nout, ctypes.byref(pol), ctypes.byref(s)),
           "qmm_splitk_plan")
    return s.value


def qmm_splitk_plan_near_equal(M: int, Kred: int, Nout: int, pol: qmm_policy) -> int:
    s = _I(0)
    _check(lib().qmm_splitk_plan_near_equal(M, Kred, Nout, ctypes.byref(pol), ctypes.byref(s)),
           "qmm_splitk_plan_near_equal")
    return s.value


def qmm_splitk_workspace_bytes(M: int, Nout: int, split: int,
                               partial_dtype: int = QMM_PARTIAL_BF16, options=None) -> int:
    if options is not None:
        return int(lib().qmm_splitk_workspace_bytes_ex(M, Nout, split, partial_dtype,
                                                        _opt(options)))
    return int(lib().qmm_splitk_workspace_bytes(M, Nout, split, partial_dtype))


def qmm_call_plan(M: int, Kred: int, Nout: int, split_req: int = 0, pol=None,
                  partial_dtype: int = QMM_PARTIAL_BF16, num_sms: int = 0, options=None,
                  with_head: bool = False):
    """(split, bm, bn) that qmm_w4a16_g128_ex would dispatch (host only);
    with_head: (split, bm, bn, head_rows), head_rows > 0 when
    QMM_SPLIT_BALANCED cuts the call."""
    s, bm, bn, hd = _I(0), _I(0), _I(0), _I(0)
    _check(lib().qmm_call_plan(M, Kred, Nout, split_req,
                               ctypes.byref(pol) if pol is not None else None, partial_dtype,
                               num_sms, _opt(options), ctypes.byref(s), ctypes.byref(bm),
                               ctypes.byref(bn), ctypes.byref(hd)), "qmm_call_plan")
    return (s.value, bm.value, bn.value, hd.value) if with_head else (s.value, bm.value, bn.value)


def qmm_call_workspace_bytes(M: int, Kred: int, Nout: int, split_req: int = 0, pol=None,
                             partial_dtype: int = QMM_PARTIAL_BF16, num_sms: int = 0,
                             options=None) -> int:
    return int(lib().qmm_call_workspace_bytes(M, Kred, Nout, split_req,
                                              ctypes.byref(pol) if pol is not None else None,
                                              partial_dtype, num_sms, _opt(options)))


def qmm_gemm_workspace_bytes(M: int, N: int, split: int) -> int:
    return int(lib().qmm_gemm_workspace_bytes(M, N, split))


# ---- device entry points -------------------------------------------------

def qmm_w4a16_g128(A: torch.Tensor, Wq: torch.Tensor, scales: torch.Tensor,
                   biases: torch.Tensor, C: torch.Tensor, split_req: int = 0,
                   pol: qmm_policy | None = None, workspace: torch.Tensor | None = None,
                   partial_dtype: int = QMM_PARTIAL_BF16, stream=None, options=None) -> int:
    """C = A @ W^T (W in the W4A16-g128 format); returns the split dispatched.
    Shapes: A [M, Kred] bf16, Wq [Nout, Kred/8] int32, scales/biases
    [Nout, Kred/128] bf16, C [M, Nout] bf16; workspace any contiguous CUDA
    tensor of at least qmm_splitk_workspace_bytes(...) bytes.  options: a
    qmm_options for this call only (qmm_w4a16_g128_ex), else the process-wide
    settings."""
    M, Kred = A.shape
    Nout = Wq.shape[0]
    g = Kred // 128
    if Wq.shape != (Nout, Kred // 8) or C.shape != (M, Nout) or \
            scales.shape != (Nout, g) or biases.shape != (Nout, g):
        raise ValueError("qmm_w4a16_g128: inconsistent shapes")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    used = _I(0)
    args = (_ptr(A, _BF16, "A"), _ptr(Wq, _WORDS, "Wq"), _ptr(scales, _BF16, "scales"),
            _ptr(biases, _BF16, "biases"), _ptr(C, _BF16, "C"), M, Kred, Nout, split_req,
            ctypes.byref(pol) if pol is not None else None, ws, ws_bytes, partial_dtype,
            _stream(stream), ctypes.byref(used))
    if options is not None:
        _check(lib().qmm_w4a16_g128_ex(*args, _opt(options)), "qmm_w4a16_g128_ex")
    else:
        rc = (_lib or lib()).qmm_w4a16_g128(*args)
        if rc != QMM_OK:
            raise QmmError(rc, "qmm_w4a16_g128")
    return used.value


def qmm_w4a16_g128_partition(A: torch.Tensor, Wq: torch.Tensor, scales: torch.Tensor,
                             biases: torch.Tensor, partials: torch.Tensor, split: int,
                             partial_dtype: int = QMM_PARTIAL_BF16, stream=None) -> None:
    """The partition kernel alone: partials [split, M, Nout] (bf16 or float32
    to match partial_dtype) receives one rounded plane per partition."""
    M, Kred = A.shape
    Nout = Wq.shape[0]
    if tuple(Wq.shape) != (Nout, Kred // 8) or \
            tuple(scales.shape) != (Nout, Kred // 128) or tuple(biases.shape) != (Nout, Kred // 128):
        raise ValueError("qmm_w4a16_g128_partition: inconsistent shapes")
    want = (torch.float32,) if partial_dtype == QMM_PARTIAL_F32 else _BF16
    rc = lib().qmm_w4a16_g128_partition(
        _dev(A, _BF16, "A"), _dev(Wq, _WORDS, "Wq"), _dev(scales, _BF16, "scales"),
        _dev(biases, _BF16, "biases"), _dev(partials, want, "partials"),
        partials.numel() * partials.element_size(), M, Kred, Nout, split, partial_dtype,
        _stream(stream))
    _check(rc, "qmm_w4a16_g128_partition")


TC_PIPELINE_FIELDS = ("issuers", "dequant_sets", "a_buffers", "weight_stage_groups",
                      "act_stage_groups", "act_stages", "weight_stages", "threads", "smem")


def qmm_tc_pipeline_config(bm: int, gpp: int, smem_limit: int = 232432) -> dict:
    """The tcgen05 kernel's pipeline shape for a tile and partition (host only)."""
    out = (_I * 9)()
    _check(lib().qmm_tc_pipeline_config(bm, gpp, smem_limit, out), "qmm_tc_pipeline_config")
    return dict(zip(TC_PIPELINE_FIELDS, list(out)))


def qmm_tc_persistent_pipeline_config(bm: int, gpp: int, smem_limit: int = 231408) -> dict:
    """The persistent grouped launch's pipeline shape (host only)."""
    out = (_I * 9)()
    _check(lib().qmm_tc_persistent_pipeline_config(bm, gpp, smem_limit, out),
           "qmm_tc_persistent_pipeline_config")
    return dict(zip(TC_PIPELINE_FIELDS, list(out)))


def qmm_static_scratch_bytes() -> int:
    return int(lib().qmm_static_scratch_bytes())


def qmm_w4a16_g128_noalloc(A: torch.Tensor, Wq: torch.Tensor, scales: torch.Tensor,
                           biases: torch.Tensor, C: torch.Tensor, split_req: int = 0,
                           pol: qmm_policy | None = None, partial_dtype: int = QMM_PARTIAL_BF16,
                           stream=None) -> int:
    """qmm_w4a16_g128 with the partial planes in the library's fixed device
    buffer (no workspace argument, no allocation); returns the split."""
    M, Kred = A.shape
    Nout = Wq.shape[0]
    if Wq.shape != (Nout, Kred // 8) or C.shape != (M, Nout) or \
            scales.shape != (Nout, Kred // 128) or biases.shape != (Nout, Kred // 128):
        raise ValueError("qmm_w4a16_g128_noalloc: inconsistent shapes")
    used = _I(0)
    rc = lib().qmm_w4a16_g128_noalloc(
        _ptr(A, _BF16, "A"), _ptr(Wq, _WORDS, "Wq"), _ptr(scales, _BF16, "scales"),
        _ptr(biases, _BF16, "biases"), _ptr(C, _BF16, "C"), M, Kred, Nout, split_req,
        ctypes.byref(pol) if pol is not None else None, partial_dtype, _stream(stream),
        ctypes.byref(used))
    _check(rc, "qmm_w4a16_g128_noalloc")
    return used.value


def qmm_splitk_reduce(partials: torch.Tensor, partial_dtype: int, split: int, M: int, Nout: int,
                      C: torch.Tensor, stream=None) -> None:
    want = (torch.float32,) if partial_dtype == QMM_PARTIAL_F32 else _BF16
    if partials.numel() < split * M * Nout or C.numel() < M * Nout:
        raise ValueError("qmm_splitk_reduce: buffers too small")
    _check(lib().qmm_splitk_reduce(_dev(partials, want, "partials"), partial_dtype, split, M, Nout,
                                   _dev(C, _BF16, "C"), _stream(stream)), "qmm_splitk_reduce")


def qmm_gemm_bf16_splitk(A: torch.Tensor, W: torch.Tensor, C: torch.Tensor, split: int,
                         workspace: torch.Tensor | None = None, stream=None) -> None:
    M, K = A.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError("qmm_gemm_bf16_splitk: inconsistent shapes")
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = ctypes.c_void_p(workspace.data_ptr()), \
            workspace.numel() * workspace.element_size()
    _check(lib().qmm_gemm_bf16_splitk(_dev(A, _BF16, "A"), _dev(W, _BF16, "W"),
                                      _dev(C, _BF16, "C"), M, N, K, split, ws, ws_bytes,
                                      _stream(stream)), "qmm_gemm_bf16_splitk")


def qmm_unpack_probe(Wq: torch.Tensor, Kred: int, q: torch.Tensor, stream=None) -> None:
    Nout = Wq.shape[0]
    if q.numel() < Nout * Kred:
        raise ValueError("qmm_unpack_probe: q too small")
    _check(lib().qmm_unpack_probe(_dev(Wq, _WORDS, "Wq"), Nout, Kred,
                                  _dev(q, (torch.uint8,), "q"), _stream(stream)),
           "qmm_unpack_probe")


def qmm_dequant_probe(Wq: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, Kred: int,
                      w: torch.Tensor, stream=None) -> None:
    Nout = Wq.shape[0]
    if w.numel() < Nout * Kred:
        raise ValueError("qmm_dequant_probe: w too small")
    _check(lib().qmm_dequant_probe(_dev(Wq, _WORDS, "Wq"), _dev(scales, _BF16, "scales"),
                                   _dev(biases, _BF16, "biases"), Nout, Kred,
                                   _dev(w, _BF16, "w"), _stream(stream)), "qmm_dequant_probe")


# ---- convenience ---------------------------------------------------------

def w4a16_matmul(A, Wq, scales, biases, split_req: int = 0, pol=None,
                 partial_dtype: int = QMM_PARTIAL_BF16, stream=None):
    """Allocate C (and the workspace the plan needs) with torch and call
    qmm_w4a16_g128.  Returns (C, split_used)."""
    M, Kred = A.shape
    Nout = Wq.shape[0]
    C = torch.empty((M, Nout), dtype=torch.bfloat16, device=A.device)
    # the workspace of the call as the library plans it, for any split_req
    # (policy, forced, QMM_SPLIT_PLANNED or QMM_SPLIT_BALANCED)
    nbytes = qmm_call_workspace_bytes(M, Kred, Nout, split_req, pol, partial_dtype)
    # zeroed: under QMM_REDUCE_FUSED the workspace's tail holds tile counters
    # that must start at zero
    ws = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=A.device) if nbytes else None
    used = qmm_w4a16_g128(A, Wq, scales, biases, C, split_req=split_req, pol=pol, workspace=ws,
                          partial_dtype=partial_dtype, stream=stream)
    return C, used


def to_device(problem: dict, device="cuda") -> dict:
    """Move a problem from split_w4a16_quantized_gb300.inputs to the GPU as the
    tensors qmm_w4a16_g128 takes."""
    import numpy as np

    def bf16(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16) \
            .to(device)

    return {
        "A": bf16(problem["A"]),
        "Wq": torch.from_numpy(np.ascontiguousarray(problem["Wq"]).view(np.int32)).to(device),
        "scales": bf16(problem["scales"]),
        "biases": bf16(problem["biases"]),
    }


# ---- streaming host activations (copy in / compute / copy out) -------------

def _host(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.bfloat16:
        raise TypeError("%s must be a host BF16 tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def stream_calls(chunks) -> "ctypes.Array":
    """chunks: sequence of dicts with host A and C (BF16, pinned to overlap) and
    device Wq, scales, biases.  Returns the qmm_stream_call array."""
    arr = (qmm_stream_call * len(chunks))()
    for i, c in enumerate(chunks):
        M, Kred = c["A"].shape
        Nout = c["Wq"].shape[0]
        if tuple(c["C"].shape) != (M, Nout):
            raise ValueError("chunk %d: C must be [M, Nout]" % i)
        arr[i] = qmm_stream_call(_host(c["A"], "A"), _host(c["C"], "C"),
                                 _dev(c["Wq"], _WORDS, "Wq").value,
                                 _dev(c["scales"], _BF16, "scales").value,
                                 _dev(c["biases"], _BF16, "biases").value, M, Kred, Nout)
    return arr


def qmm_stream_arena_bytes(calls, buffers: int) -> int:
    return int(lib().qmm_stream_arena_bytes(calls, len(calls), buffers))


def qmm_w4a16_g128_stream(calls, buffers: int, arena: torch.Tensor, stream_in=None,
                          stream_compute=None, stream_out=None):
    """Enqueue the copy-in / compute / copy-out pipeline; returns the splits used.
    Synchronize stream_out before reading the host outputs."""
    n = len(calls)
    used = (_I * n)()
    _check(lib().qmm_w4a16_g128_stream(calls, n, buffers, _dev(arena, (torch.uint8,), "arena"),
                                       arena.numel(), _stream(stream_in),
                                       _stream(stream_compute), _stream(stream_out), used),
           "qmm_w4a16_g128_stream")
    return list(used)


def qmm_overlap_schedule(n: int, buffers: int, t_load, t_comp, t_store, out_reuse=False,
                         with_events=False):
    """The pipeline's schedule model: end of the last store (and the [n, 6] events)."""
    import numpy as np
    t = [np.ascontiguousarray(np.broadcast_to(np.asarray(x, np.float64), (n,)))
         for x in (t_load, t_comp, t_store)]
    D = ctypes.POINTER(ctypes.c_double)
    T = ctypes.c_double(0.0)
    ev = np.empty((n, 6), np.float64) if with_events else None
    _check(lib().qmm_overlap_schedule(n, buffers, *(a.ctypes.data_as(D) for a in t),
                                      int(bool(out_reuse)), ctypes.byref(T),
                                      ev.ctypes.data_as(D) if ev is not None else None),
           "qmm_overlap_schedule")
    return (T.value, ev) if with_events else T.value


# ---- several independent calls in few launches ----------------------------

def group_calls(calls) -> "ctypes.Array":
    """calls: sequence of dicts of device tensors A, Wq, scales, biases, C.
    Returns the qmm_group_call array (shapes checked here)."""
    arr = (qmm_group_call * len(calls))()
    for i, c in enumerate(calls):
        M, Kred = c["A"].shape
        Nout = c["Wq"].shape[0]
        if tuple(c["Wq"].shape) != (Nout, Kred // 8) or tuple(c["C"].shape) != (M, Nout) or \
                tuple(c["scales"].shape) != (Nout, Kred // 128) or \
                tuple(c["biases"].shape) != (Nout, Kred // 128):
            raise ValueError("group call %d: inconsistent shapes" % i)
        arr[i] = qmm_group_call(_dev(c["A"], _BF16, "A").value, _dev(c["Wq"], _WORDS, "Wq").value,
                                _dev(c["scales"], _BF16, "scales").value,
                                _dev(c["biases"], _BF16, "biases").value,
                                _dev(c["C"], _BF16, "C").value, M, Kred, Nout)
    return arr


def qmm_group_workspace_bytes(calls, partial_dtype: int = QMM_PARTIAL_BF16,
                              options=None) -> int:
    if options is not None:
        return int(lib().qmm_group_workspace_bytes_ex(calls, len(calls), partial_dtype,
                                                       _opt(options)))
    return int(lib().qmm_group_workspace_bytes(calls, len(calls), partial_dtype))


def qmm_w4a16_g128_grouped(calls, workspace: torch.Tensor | None = None,
                           partial_dtype: int = QMM_PARTIAL_BF16, stream=None, options=None):
    """Every call's C with its policy split, in few launches; returns the splits."""
    n = len(calls)
    used = (_I * n)()
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _dev(workspace, (workspace.dtype,), "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    args = (calls, n, ws_ptr, ws_bytes, partial_dtype, _stream(stream), used)
    if options is not None:
        _check(lib().qmm_w4a16_g128_grouped_ex(*args, _opt(options)), "qmm_w4a16_g128_grouped_ex")
    else:
        _check(lib().qmm_w4a16_g128_grouped(*args), "qmm_w4a16_g128_grouped")
    return list(used)


# ---- paged KV cache: append, tree attention, accepted path ----------------------

QMM_CACHE_BF16, QMM_CACHE_E4M3 = 0, 1
_CACHE_DTYPES = {torch.bfloat16: QMM_CACHE_BF16, torch.float8_e4m3fn: QMM_CACHE_E4M3}
_INT32 = (torch.int32,)


def kv_cache(K: torch.Tensor, V: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
             k_scale: float = 1.0, v_scale: float = 1.0) -> qmm_kv_cache:
    """The cache of one layer: K, V [num_pages, Hkv, page_size, D] (bf16 or
    float8_e4m3fn, any strides that keep a row's D values together, both the
    same: pages of [page_size, Hkv, D] come as K.transpose(1, 2)), table int32
    [B, max_pages], lens int32 [B].  Checked once here; the tensors are kept
    alive by the result, whose pointers stay theirs."""
    if not (isinstance(K, torch.Tensor) and isinstance(V, torch.Tensor) and K.is_cuda and V.is_cuda):
        raise TypeError("K and V must be CUDA tensors")
    if K.dtype not in _CACHE_DTYPES or V.dtype != K.dtype:
        raise TypeError("K and V must both be bfloat16 or float8_e4m3fn")
    # (a dimension of one row has no stride to compare)
    if K.dim() != 4 or V.shape != K.shape or any(
            a != b and n > 1 for a, b, n in zip(K.stride(), V.stride(), K.shape)):
        raise ValueError("K and V must be [num_pages, Hkv, page_size, D] with equal strides")
    if K.stride(3) != 1:
        raise ValueError("a cache row's values must be contiguous")
    _dev(table, _INT32, "table")
    _dev(lens, _INT32, "lens")
    if table.dim() != 2 or tuple(lens.shape) != (table.shape[0],):
        raise ValueError("table must be [B, max_pages] and lens [B]")
    if len({t.get_device() for t in (K, V, table, lens)}) != 1:
        raise ValueError("the cache's tensors are on different devices")
    pages, Hkv, page, D = K.shape
    c = qmm_kv_cache(K.data_ptr(), V.data_ptr(), table.data_ptr(), lens.data_ptr(), K.stride(0),
                     K.stride(1), K.stride(2), table.shape[0], pages, page, table.shape[1], Hkv, D,
                     _CACHE_DTYPES[K.dtype], float(k_scale), float(v_scale))
    c.tensors = (K, V, table, lens)
    c.device = K.get_device()
    c.ref = ctypes.addressof(c)
    return c


def kv_caches(caches) -> "ctypes.Array":
    """The layers' caches as the array qmm_tree_accept takes."""
    if not len(caches):
        raise ValueError("at least one cache")
    arr = (qmm_kv_cache * len(caches))(*caches)
    arr.tensors = [c.tensors for c in caches]
    arr.device = caches[0].device
    if any(c.device != arr.device for c in caches):
        raise ValueError("the caches are on different devices")
    arr.n, arr.B, arr.ref = len(caches), caches[0].B, ctypes.addressof(arr)
    return arr


def rope(cos_sin: torch.Tensor | None = None, interleaved: bool = False,
         q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
         eps: float = 1e-6) -> qmm_rope:
    """Rotation by cos_sin (float32 [rows, dim], cosines then sines) and the
    optional per-head norm weights q_norm, k_norm (bf16 [D]) of qmm_kv_append."""
    rows, dim = (0, 0) if cos_sin is None else cos_sin.shape
    p = [None if t is None else _dev(t, d, n).value for t, d, n in
         ((cos_sin, (torch.float32,), "cos_sin"), (q_norm, _BF16, "q_norm"),
          (k_norm, _BF16, "k_norm"))]
    r = qmm_rope(p[0], p[1], p[2], rows, dim, int(bool(interleaved)), float(eps))
    r.tensors = (cos_sin, q_norm, k_norm)
    dims = {t.numel() for t in (q_norm, k_norm) if t is not None}
    devices = {t.get_device() for t in r.tensors if t is not None}
    if len(dims) > 1 or len(devices) > 1:
        raise ValueError("norm weights of different lengths, or tensors on different devices")
    r.D, r.device = max(dims, default=0), max(devices, default=-1)
    r.ref = ctypes.addressof(r)
    return r


def _elsewhere(device: int, tensors):
    """Report the tensor that is not on `device` (or is none), or that `device`
    is not the current one."""
    for t in tensors:
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError("expected CUDA tensors")
        if t is not None and t.get_device() != device:
            if not t.is_cuda:
                raise TypeError("expected CUDA tensors")
            raise ValueError("a tensor is not on the cache's device")
    raise ValueError("the cache's device is not the current one")


def _current(device: int) -> bool:
    """Whether `device`, where a tensor was found, is the current one: the
    kernels run there."""
    return (_cur_device or torch.cuda.current_device)() == device


def _stream_on(device: int, stream):
    """_stream for the current device, which is `device` and in use."""
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


def _heads(t: torch.Tensor, N: int, H: int, D: int, name: str) -> int:
    """The token stride of [N, H, D] bf16 rows whose heads are contiguous."""
    s0, s1, s2 = t.stride()
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be bfloat16" % name)
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    return s0 if N > 1 else H * D


def _ints(t: torch.Tensor, N: int, name: str) -> int:
    """Pointer of an int32 vector of N elements."""
    if t.dtype is not torch.int32:
        raise TypeError("%s must be int32" % name)
    if t.numel() != N or not t.is_contiguous():
        raise ValueError("%s must be contiguous, of %d elements" % (name, N))
    return t.data_ptr()


def rope_axes(axis_of_pair, axes: int | None = None) -> qmm_rope_axes:
    """The axis (0 .. axes - 1) that each rotated pair of a head turns by, one for
    each of the rope's dim / 2 pairs (qmm_kv_append_axes); axes: the positions of a
    token, None for as many as the pairs name."""
    axis = [int(a) for a in axis_of_pair]
    axes = max(axis, default=0) + 1 if axes is None else int(axes)
    if not 1 <= len(axis) <= 64 or not 1 <= axes <= 8 or min(axis) < 0 or max(axis) >= axes:
        raise ValueError("rope_axes: 1 to 64 pairs, 1 to 8 axes, each pair's among them")
    r = qmm_rope_axes(axes, (ctypes.c_uint8 * 64)(*axis))
    r.pairs, r.ref = len(axis), ctypes.addressof(r)
    return r


def _append(name: str, cache: qmm_kv_cache, q, k, v, q_out, rope, positions, cu, stream, axes=None):
    if (q is None) != (q_out is None):
        raise ValueError("%s: q and q_out come together" % name)
    device = cache.device
    if not (k.get_device() == device == v.get_device() and _current(device) and
            (q is None or q.get_device() == device == q_out.get_device()) and
            (positions is None or positions.get_device() == device) and
            (cu is None or cu.get_device() == device)):
        _elsewhere(device, (q, k, v, q_out, positions, cu))
    shape = k.shape
    N, Hkv, D = shape
    if Hkv != cache.Hkv or D != cache.D or v.shape != shape:
        raise ValueError("%s: inconsistent shapes" % name)
    Hq = qs = qos = 0
    qp = qop = None
    if q is not None:
        shape = q.shape
        Hq = shape[1]
        if shape != (N, Hq, D) or q_out.shape != shape:
            raise ValueError("%s: inconsistent shapes" % name)
        qs, qos = _heads(q, N, Hq, D, "q"), _heads(q_out, N, Hq, D, "q_out")
        qp, qop = q.data_ptr(), q_out.data_ptr()
    r = None
    if rope is not None:
        if rope.D not in (0, D) or rope.device not in (-1, device):
            raise ValueError("%s: norm weights must have D elements, and the rope's "
                             "tensors the cache's device" % name)
        r = rope.ref
    args = (cache.ref, qp, k.data_ptr(), v.data_ptr(), qop, N, Hq, qs, _heads(k, N, Hkv, D, "k"),
            _heads(v, N, Hkv, D, "v"), qos, None if cu is None else _ints(cu, cache.B + 1, "cu"))
    if axes is None:
        rc = (_lib or lib()).qmm_kv_append(
            *args, None if positions is None else _ints(positions, N, "positions"), r,
            _stream_on(device, stream))
    else:
        rc = (_lib or lib()).qmm_kv_append_axes(*args, _ints(positions, axes.axes * N, "positions"),
                                                r, axes.ref, _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, name)


def qmm_kv_append(cache: qmm_kv_cache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                  q_out: torch.Tensor | None = None, rope: qmm_rope | None = None,
                  positions: torch.Tensor | None = None, cu: torch.Tensor | None = None,
                  stream=None) -> None:
    """Rotate q [N, Hq, D] into q_out and append k, v [N, Hkv, D] (bf16; token
    strides free, so views of one fused projection do) behind the cached
    tokens.  q and q_out may both be None (only append); q_out may be q.
    positions int32 [N] and cu int32 [B + 1]: see qmm.h."""
    _append("qmm_kv_append", cache, q, k, v, q_out, rope, positions, cu, stream)


def qmm_kv_append_axes(cache: qmm_kv_cache, q: torch.Tensor | None, k: torch.Tensor,
                       v: torch.Tensor, positions: torch.Tensor, axes: qmm_rope_axes,
                       rope: qmm_rope, q_out: torch.Tensor | None = None,
                       cu: torch.Tensor | None = None, stream=None) -> None:
    """qmm_kv_append with positions int32 [axes, N], one of each axis: pair j of a
    head turns by positions[axis_of_pair[j]] (rope_axes; see qmm.h)."""
    if axes.pairs * 2 != rope.dim:
        raise ValueError("qmm_kv_append_axes: an axis for each of the rope's dim / 2 pairs")
    if positions.dim() != 2 or positions.shape[0] != axes.axes or positions.shape[1] != k.shape[0]:
        raise ValueError("qmm_kv_append_axes: positions must be [axes, N]")
    _append("qmm_kv_append_axes", cache, q, k, v, q_out, rope, positions, cu, stream, axes)


def qmm_tree_attention_workspace_bytes(cache: qmm_kv_cache, Hq: int, T: int,
                                       num_sms: int = 0) -> int:
    return int(lib().qmm_tree_attention_workspace_bytes(ctypes.byref(cache), Hq, T, num_sms))


def qmm_tree_attention(cache: qmm_kv_cache, q: torch.Tensor, O: torch.Tensor, T: int,
                       parents: torch.Tensor | None = None, cu: torch.Tensor | None = None,
                       scale: float = 0.0, workspace: torch.Tensor | None = None,
                       stream=None) -> None:
    """O [N, Hq, D] = attention of the drafted tokens q [N, Hq, D] (at most T a
    sequence, their keys already appended) over the cache; parents int32 [N]
    gives the trees, None a chain (see qmm.h)."""
    device = cache.device
    if not (q.get_device() == device == O.get_device() and _current(device) and
            (parents is None or parents.get_device() == device) and
            (cu is None or cu.get_device() == device) and
            (workspace is None or workspace.get_device() == device)):
        _elsewhere(device, (q, O, parents, cu, workspace))
    shape = q.shape
    N, Hq, D = shape
    if D != cache.D or O.shape != shape:
        raise ValueError("qmm_tree_attention: inconsistent shapes")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    rc = (_lib or lib()).qmm_tree_attention(
        cache.ref, q.data_ptr(), _heads(q, N, Hq, D, "q"), _ptr(O, _BF16, "O"), N, T, Hq,
        None if cu is None else _ints(cu, cache.B + 1, "cu"),
        None if parents is None else _ints(parents, N, "parents"), scale, ws, ws_bytes,
        _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_tree_attention")


def prefix(table: torch.Tensor, lens: torch.Tensor, first: torch.Tensor) -> qmm_prefix:
    """Prefixes that runs of a batch's sequences share: table int32 [G, max_pages],
    lens int32 [G], first int32 [G + 1] (sequences first[g] .. first[g + 1] - 1 share
    prefix g).  Checked once here; the tensors are kept alive by the result."""
    for t, n in ((table, "table"), (lens, "lens"), (first, "first")):
        _dev(t, _INT32, n)
    if table.dim() != 2 or tuple(lens.shape) != (table.shape[0],) or \
            tuple(first.shape) != (table.shape[0] + 1,):
        raise ValueError("table must be [G, max_pages], lens [G] and first [G + 1]")
    if len({t.get_device() for t in (table, lens, first)}) != 1:
        raise ValueError("the prefixes' tensors are on different devices")
    p = qmm_prefix(table.data_ptr(), lens.data_ptr(), first.data_ptr(), *table.shape)
    p.tensors = (table, lens, first)
    p.device = table.get_device()
    p.ref = ctypes.addressof(p)
    return p


def qmm_prefix_attention_workspace_bytes(cache: qmm_kv_cache, Hq: int, N: int, T: int,
                                         num_sms: int = 0) -> int:
    return int(lib().qmm_prefix_attention_workspace_bytes(ctypes.byref(cache), Hq, N, T, num_sms))


def qmm_prefix_attention(cache: qmm_kv_cache, prefix: qmm_prefix, q: torch.Tensor,
                         O: torch.Tensor, T: int, parents: torch.Tensor | None = None,
                         cu: torch.Tensor | None = None, scale: float = 0.0,
                         workspace: torch.Tensor | None = None, stream=None) -> None:
    """qmm_tree_attention of a batch whose sequences also see the prefix that they
    share (prefix()), in front of their own slots (see qmm.h)."""
    device = cache.device
    if not (q.get_device() == device == O.get_device() and _current(device) and
            (parents is None or parents.get_device() == device) and
            (cu is None or cu.get_device() == device) and
            (workspace is None or workspace.get_device() == device)):
        _elsewhere(device, (q, O, parents, cu, workspace))
    if prefix.device != device:
        raise ValueError("the prefixes are not on the cache's device")
    shape = q.shape
    N, Hq, D = shape
    if D != cache.D or O.shape != shape:
        raise ValueError("qmm_prefix_attention: inconsistent shapes")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    rc = (_lib or lib()).qmm_prefix_attention(
        cache.ref, prefix.ref, q.data_ptr(), _heads(q, N, Hq, D, "q"), _ptr(O, _BF16, "O"), N, T,
        Hq, None if cu is None else _ints(cu, cache.B + 1, "cu"),
        None if parents is None else _ints(parents, N, "parents"), scale, ws, ws_bytes,
        _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_prefix_attention")


def qmm_tree_accept(caches, tokens: torch.Tensor, targets: torch.Tensor, T: int,
                    path: torch.Tensor, count: torch.Tensor, next: torch.Tensor | None = None,
                    new_lens: torch.Tensor | None = None, parents: torch.Tensor | None = None,
                    cu: torch.Tensor | None = None, stream=None) -> None:
    """Follow targets down the drafted trees (tokens, parents int32 [N]) and
    move the accepted rows in every cache of `caches` (kv_caches()).  path
    int32 [B, T], count, next and new_lens int32 [B] (see qmm.h)."""
    device, B = caches.device, caches.B
    if not (tokens.get_device() == device == targets.get_device() and _current(device) and
            path.get_device() == device == count.get_device() and
            (next is None or next.get_device() == device) and
            (new_lens is None or new_lens.get_device() == device) and
            (parents is None or parents.get_device() == device) and
            (cu is None or cu.get_device() == device)):
        _elsewhere(device, (tokens, targets, path, count, next, new_lens, parents, cu))
    N = tokens.numel()
    rc = (_lib or lib()).qmm_tree_accept(
        caches.ref, caches.n, _ints(tokens, N, "tokens"), _ints(targets, N, "targets"),
        None if parents is None else _ints(parents, N, "parents"),
        None if cu is None else _ints(cu, B + 1, "cu"), N, T, _ints(path, B * T, "path"),
        _ints(count, B, "count"), None if next is None else _ints(next, B, "next"),
        None if new_lens is None else _ints(new_lens, B, "new_lens"), _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_tree_accept")


def _mass(t: torch.Tensor, layers: int, cache: qmm_kv_cache, name: str):
    """Layer and row strides of weights [layers, B, Hkv, S] (one layer: [B, Hkv, S]
    too), S at least the slots of a sequence's table."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.float32:
        raise TypeError("%s must be float32" % name)
    if layers == 1 and len(shape) == 3:
        shape, stride = (1, *shape), (0, *stride)
    if len(shape) != 4 or shape[:3] != (layers, cache.B, cache.Hkv) or \
            shape[3] < cache.max_pages * cache.page_size:
        raise ValueError("%s must be [layers, B, Hkv, S], S at least max_pages * page_size" % name)
    # (a dimension of one row has no stride)
    row = stride[2] if cache.Hkv > 1 else (stride[1] if cache.B > 1 else (shape[3] + 3) // 4 * 4)
    if stride[3] != 1 or (cache.B > 1 and stride[1] != cache.Hkv * row):
        raise ValueError("%s: a layer's rows must be evenly spaced, their values contiguous" % name)
    return stride[0] if layers > 1 else cache.B * cache.Hkv * row, row


def qmm_scored_attention_workspace_bytes(cache: qmm_kv_cache, Hq: int, T: int,
                                         num_sms: int = 0) -> int:
    return int(lib().qmm_scored_attention_workspace_bytes(ctypes.byref(cache), Hq, T, num_sms))


def qmm_scored_attention(cache: qmm_kv_cache, q: torch.Tensor, O: torch.Tensor, T: int,
                         mass: torch.Tensor, decay: float = 1.0, cu: torch.Tensor | None = None,
                         scale: float = 0.0, workspace: torch.Tensor | None = None,
                         stream=None) -> None:
    """qmm_tree_attention of a chain that also adds each slot's softmax weights to
    mass, float32 [B, Hkv, S], whose old sums count `decay` times (see qmm.h)."""
    device = cache.device
    if not (q.get_device() == device == O.get_device() and _current(device) and
            mass.get_device() == device and (cu is None or cu.get_device() == device) and
            (workspace is None or workspace.get_device() == device)):
        _elsewhere(device, (q, O, mass, cu, workspace))
    shape = q.shape
    N, Hq, D = shape
    if D != cache.D or O.shape != shape:
        raise ValueError("qmm_scored_attention: inconsistent shapes")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    rc = (_lib or lib()).qmm_scored_attention(
        cache.ref, q.data_ptr(), _heads(q, N, Hq, D, "q"), _ptr(O, _BF16, "O"), N, T, Hq,
        None if cu is None else _ints(cu, cache.B + 1, "cu"), scale, mass.data_ptr(),
        _mass(mass, 1, cache, "mass")[1], decay, ws, ws_bytes, _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_scored_attention")


def qmm_kv_evict(caches, mass: torch.Tensor, keep: int, kept: torch.Tensor,
                 new_lens: torch.Tensor, sinks: int = 0, recent: int = 0,
                 mass_out: torch.Tensor | None = None, stream=None) -> None:
    """Bring every sequence of `caches` (kv_caches()) back to `keep` slots: the
    first `sinks`, the last `recent` and the heaviest others by mass, float32 [n,
    B, Hkv, S], whose values move along into mass_out (None: mass itself).  kept
    int32 [n, B, Hkv, keep] and new_lens int32 [B] are written (see qmm.h)."""
    device, B, n = caches.device, caches.B, caches.n
    mass_out = mass if mass_out is None else mass_out
    if not (mass.get_device() == device == mass_out.get_device() and _current(device) and
            kept.get_device() == device == new_lens.get_device()):
        _elsewhere(device, (mass, mass_out, kept, new_lens))
    c = caches[0]
    strides = _mass(mass, n, c, "mass")
    if mass_out is not mass and _mass(mass_out, n, c, "mass_out") != strides:
        raise ValueError("qmm_kv_evict: mass and mass_out must have the same strides")
    rc = (_lib or lib()).qmm_kv_evict(
        caches.ref, n, mass.data_ptr(), mass_out.data_ptr(), *strides, keep, sinks, recent,
        _ints(kept, n * B * c.Hkv * keep, "kept"), _ints(new_lens, B, "new_lens"),
        _stream_on(device, stream))
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_kv_evict")


# ---- split-KV decode attention ---------------------------------------------

def qmm_decode_attention_splits(B: int, Hq: int, Hkv: int, Lmax: int, num_sms: int = 0) -> int:
    s = _I(0)
    _check(lib().qmm_decode_attention_splits(B, Hq, Hkv, Lmax, num_sms, ctypes.byref(s)),
           "qmm_decode_attention_splits")
    return s.value


def qmm_decode_attention_workspace_bytes(B: int, Hq: int, D: int, splits: int) -> int:
    return int(lib().qmm_decode_attention_workspace_bytes(B, Hq, D, splits))


def qmm_decode_attention(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lens: torch.Tensor,
                         O: torch.Tensor, scale: float = 0.0, splits_req: int = 0,
                         workspace: torch.Tensor | None = None, stream=None) -> int:
    """O = split-KV decode attention (see qmm.h); returns the split used.
    q [B, Hq, D], K/V [B, Hkv, Lmax, D] bf16, lens int32 [B] (device), O [B, Hq, D] bf16."""
    B, Hq, D = q.shape
    _, Hkv, Lmax, _ = K.shape
    if tuple(K.shape) != (B, Hkv, Lmax, D) or tuple(V.shape) != tuple(K.shape) or \
            tuple(O.shape) != (B, Hq, D) or tuple(lens.shape) != (B,):
        raise ValueError("qmm_decode_attention: inconsistent shapes")
    used = _I(0)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _dev(workspace, (workspace.dtype,), "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().qmm_decode_attention(_dev(q, _BF16, "q"), _dev(K, _BF16, "K"),
                                      _dev(V, _BF16, "V"), _dev(lens, (torch.int32,), "lens"),
                                      _dev(O, _BF16, "O"), B, Hq, Hkv, Lmax, D, float(scale),
                                      splits_req, ws_ptr, ws_bytes, _stream(stream),
                                      ctypes.byref(used)), "qmm_decode_attention")
    return used.value


def attention_to_device(problem: dict, device="cuda") -> dict:
    """Upload an inputs.make_attention problem: q, K, V as bf16, lens as int32."""
    def bf16(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16) \
            .to(device)
    return {"q": bf16(problem["q"]), "K": bf16(problem["K"]), "V": bf16(problem["V"]),
            "lens": torch.from_numpy(problem["lens"]).to(device)}
