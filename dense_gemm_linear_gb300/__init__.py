"""GB300 (sm_103a) dense linear-layer GEMM: C = A . B^T in bf16, E4M3 and MXFP4.

Python binding of the C ABI in ``include/dgl.h``.  Functions named ``dgl_*``
marshal plain integers/pointers into the library one to one; the ``gemm_*``
helpers take torch CUDA tensors, allocate the output with torch when none is
given, and call the same entry points on torch's current stream.  Every step
of the computation runs in the library's CUDA kernels; if the library is
missing, loading raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import metrics  # noqa: F401  (pure-Python metric helpers)

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "_build", "libdgl.so")

DGL_OK = 0
DGL_ERR_ARG = -1
DGL_ERR_ALIGN = -2
DGL_ERR_SHAPE = -3
DGL_ERR_UNSUPPORTED = -4
DGL_ERR_CUDA = -5
DGL_ERR_TIMEOUT = -6

OUT_BF16 = 0
OUT_F32 = 1
DTYPE_BF16 = 0
DTYPE_E4M3 = 1
DTYPE_MXFP4 = 2
DTYPE_W4A8 = 3
PATH_TC = 0
PATH_DECODE = 1
PATH_EMPTY = 2
ACT_NONE = 0
ACT_GELU = 1
ACT_SILU = 2
K_MAJOR = 0
MN_MAJOR = 1

EXPORTED = ["dgl_gemm_bf16", "dgl_gemm_fp8", "dgl_gemm_planned", "dgl_plan", "dgl_tile_metrics",
            "dgl_device_status", "dgl_status_string", "dgl_version", "dgl_gemm_noalloc", "dgl_linear",
            "dgl_plan_linear", "dgl_gemm_bf16_ex", "dgl_gemm_mxfp4", "dgl_shutdown", "dgl_gemm_w4a8",
            "dgl_gemm_batch", "dgl_head_workspace", "dgl_linear_xent", "dgl_linear_distill"]

DISTILL_MAX_K = 128


class PlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("stages", ctypes.c_int32), ("cta_group", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("num_tiles", ctypes.c_int32), ("tile_eff", ctypes.c_double),
                ("wq_eff", ctypes.c_double), ("dim_eff", ctypes.c_double), ("est_us", ctypes.c_double),
                ("stream_k", ctypes.c_int32), ("split_tail", ctypes.c_int32), ("k_group", ctypes.c_int32)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class GemmDesc(ctypes.Structure):
    """One GEMM of dgl_gemm_batch (the C struct dgl_gemm_desc)."""
    _fields_ = [("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("scale_a", ctypes.c_void_p), ("scale_b", ctypes.c_void_p),
                ("C", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("m_valid", ctypes.c_int64), ("n_valid", ctypes.c_int64)]


class HeadDesc(ctypes.Structure):
    """Arguments of the head losses (the C struct dgl_head_desc)."""
    _fields_ = [("T", ctypes.c_int64), ("V", ctypes.c_int64), ("d", ctypes.c_int64), ("X", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("loss", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("dX", ctypes.c_void_p), ("lddx", ctypes.c_int64),
                ("dW", ctypes.c_void_p), ("lddw", ctypes.c_int64), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_int64), ("logit_scale", ctypes.c_float), ("dw_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32)]


class DglError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lib = None


def load_library(path: str | None = None):
    """Load libdgl.so (build it first with ``_build.build()``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with dense_gemm_linear_gb300._build.build()")
    lib = ctypes.CDLL(p)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.dgl_gemm_bf16.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    lib.dgl_gemm_bf16.restype = i32
    lib.dgl_gemm_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    lib.dgl_gemm_fp8.restype = i32
    lib.dgl_gemm_planned.argtypes = [i32, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32,
                                     ctypes.POINTER(PlanInfo), vp]
    lib.dgl_gemm_planned.restype = i32
    lib.dgl_gemm_noalloc.argtypes = [i32, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    lib.dgl_gemm_noalloc.restype = i32
    lib.dgl_linear.argtypes = [i32, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, i32,
                               ctypes.POINTER(PlanInfo), vp]
    lib.dgl_linear.restype = i32
    lib.dgl_plan_linear.argtypes = [i32, i64, i64, i64, i32, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.dgl_plan_linear.restype = i32
    lib.dgl_gemm_bf16_ex.argtypes = [i32, i32, vp, i64, vp, i64, vp, i64, i64, i64, i64, i32,
                                     ctypes.POINTER(PlanInfo), vp]
    lib.dgl_gemm_bf16_ex.restype = i32
    lib.dgl_gemm_w4a8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    lib.dgl_gemm_w4a8.restype = i32
    lib.dgl_gemm_mxfp4.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    lib.dgl_gemm_mxfp4.restype = i32
    lib.dgl_gemm_batch.argtypes = [ctypes.POINTER(GemmDesc), i32, vp]
    lib.dgl_gemm_batch.restype = i32
    lib.dgl_head_workspace.argtypes = [ctypes.POINTER(HeadDesc), i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.dgl_head_workspace.restype = i32
    lib.dgl_linear_xent.argtypes = [ctypes.POINTER(HeadDesc), vp, i64, vp]
    lib.dgl_linear_xent.restype = i32
    lib.dgl_linear_distill.argtypes = [ctypes.POINTER(HeadDesc), vp, vp, vp, i32, ctypes.c_float, vp]
    lib.dgl_linear_distill.restype = i32
    lib.dgl_plan.argtypes = [i32, i64, i64, i64, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.dgl_plan.restype = i32
    lib.dgl_tile_metrics.argtypes = [i64, i64, i32, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.dgl_tile_metrics.restype = i32
    lib.dgl_shutdown.argtypes = []
    lib.dgl_shutdown.restype = i32
    lib.dgl_device_status.argtypes = [vp]
    lib.dgl_device_status.restype = i32
    lib.dgl_status_string.argtypes = [i32]
    lib.dgl_status_string.restype = ctypes.c_char_p
    lib.dgl_version.argtypes = []
    lib.dgl_version.restype = i32
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().dgl_status_string(status).decode()
    except ImportError:
        return "library not loaded"


def _check(status: int, where: str):
    if status != DGL_OK:
        raise DglError(status, where)


# ---------------------------------------------------------------- raw C-ABI calls
def dgl_gemm_bf16(A, B, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, stream=0) -> int:
    return load_library().dgl_gemm_bf16(A, B, C, M, N, K, m_valid, n_valid, out_dtype, stream)


def dgl_gemm_fp8(A, B, sa, sb, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, stream=0) -> int:
    return load_library().dgl_gemm_fp8(A, B, sa, sb, C, M, N, K, m_valid, n_valid, out_dtype, stream)


def gemm_descs(items):
    """A ctypes array of GemmDesc from dicts (or GemmDesc instances) for dgl_gemm_batch."""
    arr = (GemmDesc * len(items))()
    for i, it in enumerate(items):
        arr[i] = it if isinstance(it, GemmDesc) else GemmDesc(**it)
    return arr


def dgl_gemm_batch(items, stream=0) -> int:
    """Independent GEMMs back to back on one stream (see dgl_gemm_batch in dgl.h); items: GemmDesc array or list."""
    arr = items if isinstance(items, ctypes.Array) else gemm_descs(items)
    return load_library().dgl_gemm_batch(arr, len(arr), stream)


def dgl_gemm_mxfp4(A, B, sfa, sfb, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, stream=0) -> int:
    """Block-scaled FP4: A [m][K/2], B [n][K/2] packed E2M1 bytes; sfa [m][K/32], sfb [n][K/32] E8M0 bytes."""
    return load_library().dgl_gemm_mxfp4(A, B, sfa, sfb, C, M, N, K, m_valid, n_valid, out_dtype, stream)


def dgl_gemm_w4a8(A, B, sa, sb, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, stream=0) -> int:
    """E4M3 A [m][K] x packed E2M1 B [n][K/2] (two codes a byte), fp32 scales sa [m], sb [n]."""
    return load_library().dgl_gemm_w4a8(A, B, sa, sb, C, M, N, K, m_valid, n_valid, out_dtype, stream)


def dgl_gemm_planned(dtype, A, B, sa, sb, C, M, N, K, m_valid, n_valid, out_dtype, plan: PlanInfo,
                     stream=0) -> int:
    return load_library().dgl_gemm_planned(dtype, A, B, sa, sb, C, M, N, K, m_valid, n_valid, out_dtype,
                                           ctypes.byref(plan), stream)


def dgl_gemm_noalloc(dtype, A, B, sa, sb, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, stream=0) -> int:
    """The GEMM that allocates no device memory (stream-K partials in a fixed device array)."""
    return load_library().dgl_gemm_noalloc(dtype, A, B, sa, sb, C, M, N, K, m_valid, n_valid, out_dtype, stream)


def dgl_linear(dtype, A, B, sa, sb, bias, C, M, N, K, m_valid=0, n_valid=0, out_dtype=OUT_BF16, act=0, gated=0,
               plan: PlanInfo | None = None, stream=0) -> int:
    """Linear layer act(A . B^T + bias), or the gated form (see include/dgl.h)."""
    return load_library().dgl_linear(dtype, A, B, sa, sb, bias, C, M, N, K, m_valid, n_valid, out_dtype, act, gated,
                                     ctypes.byref(plan) if plan is not None else None, stream)


def dgl_gemm_bf16_ex(a_major, b_major, A, lda, B, ldb, C, ldc, m, n, K, out_dtype=OUT_BF16,
                     plan: PlanInfo | None = None, stream=0) -> int:
    """bf16 GEMM with K-major or MN-major operands and explicit pitches (see include/dgl.h)."""
    return load_library().dgl_gemm_bf16_ex(a_major, b_major, A, lda, B, ldb, C, ldc, m, n, K, out_dtype,
                                           ctypes.byref(plan) if plan is not None else None, stream)


def dgl_head_workspace(head: HeadDesc, k=0) -> tuple[int, int]:
    """(smallest accepted, largest useful) workspace bytes of a head loss."""
    low, best = ctypes.c_int64(), ctypes.c_int64()
    _check(load_library().dgl_head_workspace(ctypes.byref(head), k, ctypes.byref(low), ctypes.byref(best)),
           "dgl_head_workspace")
    return low.value, best.value


def dgl_linear_xent(head: HeadDesc, target, ignore_index=-100, stream=0) -> int:
    """Softmax cross entropy of a linear head (see include/dgl.h)."""
    return load_library().dgl_linear_xent(ctypes.byref(head), target, ignore_index, stream)


def dgl_linear_distill(head: HeadDesc, indices, logits, teacher_lse, k, temperature=1.0, stream=0) -> int:
    """Distillation of a linear head from a teacher's top logits (see include/dgl.h)."""
    return load_library().dgl_linear_distill(ctypes.byref(head), indices, logits, teacher_lse, k, temperature, stream)


def dgl_plan(dtype, m, n, K, out_dtype=OUT_BF16, num_sms=0) -> PlanInfo:
    info = PlanInfo()
    _check(load_library().dgl_plan(dtype, m, n, K, out_dtype, num_sms, ctypes.byref(info)), "dgl_plan")
    return info


def dgl_plan_linear(dtype, m, n, K, out_dtype=OUT_BF16, gated=0, num_sms=0) -> PlanInfo:
    info = PlanInfo()
    _check(load_library().dgl_plan_linear(dtype, m, n, K, out_dtype, int(gated), num_sms, ctypes.byref(info)),
           "dgl_plan_linear")
    return info


def dgl_tile_metrics(m, n, tile_m, tile_n, num_units) -> PlanInfo:
    info = PlanInfo()
    _check(load_library().dgl_tile_metrics(m, n, tile_m, tile_n, num_units, ctypes.byref(info)),
           "dgl_tile_metrics")
    return info


def dgl_device_status(stream=0) -> int:
    return load_library().dgl_device_status(stream)


def dgl_shutdown() -> int:
    """Free the library's workspaces and caches on the current device (see include/dgl.h)."""
    return load_library().dgl_shutdown()


def dgl_version() -> int:
    return load_library().dgl_version()


# ---------------------------------------------------------------- torch helpers
def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check_operand(t, name, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) != t.shape[1]:
        raise ValueError(f"{name} must be a contiguous 2-D tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _out_tensor(out, m, n, out_dtype, device):
    import torch
    tdt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if out is None:
        return torch.empty((m, n), dtype=tdt, device=device), n, m
    if out.dtype != tdt or out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be a 2-D row-major tensor of the output dtype")
    if out.shape[0] < m or out.stride(0) < n:
        raise ValueError("out is smaller than the valid region")
    return out, out.stride(0), out.shape[0]


def gemm_bf16(A, B, out=None, *, out_dtype=OUT_BF16, stream=None, plan: PlanInfo | None = None):
    """C = A . B^T for bf16 A [m, K], B [n, K] (CUDA tensors); returns C [m, n] (or `out`)."""
    import torch
    _check_operand(A, "A", torch.bfloat16)
    _check_operand(B, "B", torch.bfloat16)
    m, K = A.shape
    n, K2 = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    C, ldc, rows = _out_tensor(out, m, n, out_dtype, A.device)
    s = _stream_handle(stream)
    if plan is None:
        st = dgl_gemm_bf16(A.data_ptr(), B.data_ptr(), C.data_ptr(), rows, ldc, K, m, n, out_dtype, s)
    else:
        st = dgl_gemm_planned(DTYPE_BF16, A.data_ptr(), B.data_ptr(), None, None, C.data_ptr(), rows, ldc, K,
                              m, n, out_dtype, plan, s)
    _check(st, "dgl_gemm_bf16")
    return C


def gemm_fp8(A, B, sa, sb, out=None, *, out_dtype=OUT_BF16, stream=None, plan: PlanInfo | None = None):
    """C = (A . B^T) * sa[:, None] * sb[None, :] for E4M3 A [m, K], B [n, K]; fp32 scales."""
    import torch
    _check_operand(A, "A", torch.float8_e4m3fn)
    _check_operand(B, "B", torch.float8_e4m3fn)
    m, K = A.shape
    n, K2 = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    for name, s_, length in (("sa", sa, m), ("sb", sb, n)):
        if s_.dtype != torch.float32 or not s_.is_cuda or s_.numel() != length or not s_.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of length {length}")
    C, ldc, rows = _out_tensor(out, m, n, out_dtype, A.device)
    s = _stream_handle(stream)
    if plan is None:
        st = dgl_gemm_fp8(A.data_ptr(), B.data_ptr(), sa.data_ptr(), sb.data_ptr(), C.data_ptr(), rows, ldc, K,
                          m, n, out_dtype, s)
    else:
        st = dgl_gemm_planned(DTYPE_E4M3, A.data_ptr(), B.data_ptr(), sa.data_ptr(), sb.data_ptr(),
                              C.data_ptr(), rows, ldc, K, m, n, out_dtype, plan, s)
    _check(st, "dgl_gemm_fp8")
    return C


def gemm_mxfp4(A, B, sfa, sfb, K, out=None, *, out_dtype=OUT_BF16, stream=None):
    """C = sum_k 2^(sfa - 127) a * 2^(sfb - 127) b over E2M1 elements (MXFP4).

    A [m, K/2] and B [n, K/2] are uint8 CUDA tensors of packed E2M1 codes
    (element 2t in the low four bits of byte t); sfa [m, K/32] and sfb
    [n, K/32] are uint8 E8M0 scales, one per 32 elements of K.  K is passed
    explicitly (two elements per byte).  Returns C [m, n].
    """
    import torch
    m, n = A.shape[0], B.shape[0]
    for name, t, shape in (("A", A, (m, K // 2)), ("B", B, (n, K // 2)), ("sfa", sfa, (m, K // 32)),
                           ("sfb", sfb, (n, K // 32))):
        if t.dtype != torch.uint8 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor of shape {shape}")
    C, ldc, rows = _out_tensor(out, m, n, out_dtype, A.device)
    st = dgl_gemm_mxfp4(A.data_ptr(), B.data_ptr(), sfa.data_ptr(), sfb.data_ptr(), C.data_ptr(), rows, ldc, K, m,
                        n, out_dtype, _stream_handle(stream))
    _check(st, "dgl_gemm_mxfp4")
    return C


def gemm_w4a8(A, B, sa, sb, K, out=None, *, out_dtype=OUT_BF16, stream=None):
    """C = (A . B^T) * sa[:, None] * sb[None, :] for E4M3 A [m, K] and E2M1 B.

    A is a float8_e4m3fn (or uint8) CUDA tensor [m, K]; B a uint8 CUDA tensor
    [n, K/2] of packed E2M1 codes (element 2t in the low four bits of byte t);
    sa [m], sb [n] fp32.  K is passed explicitly.  Returns C [m, n].
    """
    import torch
    m, n = A.shape[0], B.shape[0]
    if A.dtype not in (torch.float8_e4m3fn, torch.uint8) or not A.is_cuda or tuple(A.shape) != (m, K) \
            or not A.is_contiguous():
        raise ValueError(f"A must be a contiguous E4M3 CUDA tensor of shape {(m, K)}")
    if B.dtype != torch.uint8 or not B.is_cuda or tuple(B.shape) != (n, K // 2) or not B.is_contiguous():
        raise ValueError(f"B must be a contiguous uint8 CUDA tensor of shape {(n, K // 2)}")
    for name, s_, length in (("sa", sa, m), ("sb", sb, n)):
        if s_.dtype != torch.float32 or not s_.is_cuda or s_.numel() != length or not s_.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of length {length}")
    C, ldc, rows = _out_tensor(out, m, n, out_dtype, A.device)
    st = dgl_gemm_w4a8(A.data_ptr(), B.data_ptr(), sa.data_ptr(), sb.data_ptr(), C.data_ptr(), rows, ldc, K, m, n,
                       out_dtype, _stream_handle(stream))
    _check(st, "dgl_gemm_w4a8")
    return C


def plan(dtype, m, n, K, out_dtype=OUT_BF16, num_sms=0) -> dict:
    return dgl_plan(dtype, m, n, K, out_dtype, num_sms).as_dict()


def device_status(stream=None) -> int:
    return dgl_device_status(_stream_handle(stream))


def build() -> str:
    from ._build import build as _b
    return _b()


def linear(A, B, bias=None, out=None, *, act=ACT_NONE, gated=False, sa=None, sb=None, out_dtype=OUT_BF16,
           stream=None, plan: PlanInfo | None = None):
    """Linear layer with a fused epilogue: act(A . B^T + bias), or with
    gated=True act(A . Bg^T + bg) * (A . Bu^T + bu) for B = [Bg; Bu] (2n rows).

    A [m, K] and B are bf16 (or E4M3 with fp32 scales sa [m], sb [rows of B]);
    bias is fp32 with one entry per row of B, or None.  Returns C [m, n].
    """
    import torch
    e4m3 = A.dtype == torch.float8_e4m3fn
    want = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    _check_operand(A, "A", want)
    _check_operand(B, "B", want)
    m, K = A.shape
    rows_b, K2 = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    if gated and rows_b % 2:
        raise ValueError("a gated layer's B holds 2n rows: gate rows, then up rows")
    n = rows_b // 2 if gated else rows_b
    vecs = [("bias", bias, rows_b)] + ([("sa", sa, m), ("sb", sb, rows_b)] if e4m3 else [])
    for name, v, length in vecs:
        if v is None and name == "bias":
            continue
        if v is None or v.dtype != torch.float32 or not v.is_cuda or v.numel() != length or not v.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of length {length}")
    C, ldc, rows = _out_tensor(out, m, n, out_dtype, A.device)
    st = dgl_linear(DTYPE_E4M3 if e4m3 else DTYPE_BF16, A.data_ptr(), B.data_ptr(),
                    sa.data_ptr() if e4m3 else None, sb.data_ptr() if e4m3 else None,
                    bias.data_ptr() if bias is not None else None, C.data_ptr(), rows, ldc, K, m, n, out_dtype,
                    int(act), int(bool(gated)), plan, _stream_handle(stream))
    _check(st, "dgl_linear")
    return C



# ---------------------------------------------------------------- losses of a linear head
def _rows(t, name, dtype, shape):
    """Checks a CUDA matrix of `shape` whose rows are contiguous; returns its row pitch in elements."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    pitch, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return pitch if shape[0] > 1 else shape[1]


def _vector(t, name, dtype, shape):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")


@functools.lru_cache(maxsize=256)
def _head_workspace_bytes(T, V, d, grad, dX, dW, dw_dtype, k):
    h = HeadDesc(T=T, V=V, d=d, grad=grad, dX=dX, dW=dW, dw_dtype=dw_dtype)
    return max(1, dgl_head_workspace(h, k)[1])


def _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, stream, k, call, where):
    import torch
    if not isinstance(X, torch.Tensor) or X.dim() != 2 or not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise TypeError("X and W must be 2-D CUDA tensors")
    T, d = X.shape
    V = W.shape[0]
    ldx = _rows(X, "X", torch.bfloat16, (T, d))
    ldw = _rows(W, "W", torch.bfloat16, (V, d))
    if stream is not None:
        # buffers made here belong to the stream that uses them, so the
        # allocator hands them out again only after its work
        with torch.cuda.stream(stream):
            return _head_on(X, W, T, V, d, ldx, ldw, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate,
                            workspace, stream.cuda_stream, k, call, where)
    return _head_on(X, W, T, V, d, ldx, ldw, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace,
                    torch._C._cuda_getCurrentRawStream(X.device.index), k, call, where)


def _head_on(X, W, T, V, d, ldx, ldw, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, s, k,
             call, where):
    import torch
    device = X.device
    loss = torch.empty(T, dtype=torch.float32, device=device)
    lse = torch.empty(T, dtype=torch.float32, device=device)
    dX = None
    p_grad = p_dx = p_dw = lddw = 0
    dw_type = OUT_BF16
    if grad is not None:
        _vector(grad, "grad", torch.float32, (T,))
        if not (need_dx or need_dw):
            raise ValueError("a call with grad computes dX, dW or both")
        p_grad = grad.data_ptr()
        if need_dx:
            dX = torch.empty((T, d), dtype=torch.bfloat16, device=device)
            p_dx = dX.data_ptr()
        if need_dw:
            if dW is None:
                if accumulate:
                    raise ValueError("accumulate adds to the fp32 dW that is passed in")
                dW = torch.empty((V, d), dtype=torch.float32 if dw_dtype == OUT_F32 else torch.bfloat16, device=device)
                lddw = d
            else:
                if dW.dtype not in (torch.float32, torch.bfloat16):
                    raise TypeError(f"dW must be fp32 or bf16, got {dW.dtype}")
                lddw = _rows(dW, "dW", dW.dtype, (V, d))
            dw_type = OUT_F32 if dW.dtype == torch.float32 else OUT_BF16
            p_dw = dW.data_ptr()
    if not need_dw or grad is None:
        if dW is not None or accumulate:
            raise ValueError("dW needs grad, the losses' upstream gradient, and need_dw")
    if workspace is None:
        workspace = torch.empty(_head_workspace_bytes(T, V, d, bool(p_grad), bool(p_dx), bool(p_dw), dw_type, k),
                                dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    h = HeadDesc(T, V, d, X.data_ptr(), ldx, W.data_ptr(), ldw, loss.data_ptr(), lse.data_ptr(), p_grad, p_dx, d, p_dw,
                 lddw, workspace.data_ptr(), workspace.nbytes, logit_scale, dw_type, int(bool(accumulate)))
    _check(call(h, s), where)
    if grad is None:
        return loss, lse
    return loss, lse, dX, dW


def linear_cross_entropy(X, W, target, grad=None, *, ignore_index=-100, logit_scale=1.0, need_dx=True, need_dw=True,
                         dW=None, dw_dtype=OUT_BF16, accumulate=False, workspace=None, stream=None):
    """Softmax cross entropy of the head z = logit_scale X . W^T, without keeping the logits.

    X [T, d], W [V, d] bf16 (rows may be strided), target int64 [T].  Returns
    (loss, lse), fp32 [T] each.  With grad, fp32 [T], the gradient of the
    final scalar by each loss (1 / tokens for a mean), returns (loss, lse, dX,
    dW): dX bf16, dW bf16 or fp32 (dw_dtype, or the type of the dW passed in;
    accumulate adds to an fp32 dW).  workspace: a CUDA buffer of at least
    dgl_head_workspace bytes, made when None.
    """
    import torch
    _vector(target, "target", torch.int64, (X.shape[0],))
    return _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, stream, 0,
                 lambda h, s: dgl_linear_xent(h, target.data_ptr(), ignore_index, s), "dgl_linear_xent")


def linear_distill(X, W, indices, logits, grad=None, *, temperature=1.0, teacher_lse=None, logit_scale=1.0,
                   need_dx=True, need_dw=True, dW=None, dw_dtype=OUT_BF16, accumulate=False, workspace=None,
                   stream=None):
    """Distillation of the head z = logit_scale X . W^T from a teacher's top logits.

    indices int64 [T, k] (negative: absent) and logits fp32 [T, k] are the
    teacher's; loss_t is the Kullback-Leibler divergence of the student's
    softmax(z / temperature) from the teacher's distribution over the entries
    (with teacher_lse, fp32 [T], from its share of the whole vocabulary's).
    Otherwise as linear_cross_entropy.
    """
    import torch
    T = X.shape[0]
    k = indices.shape[1] if indices.dim() == 2 else 0
    if not 1 <= k <= DISTILL_MAX_K:
        raise ValueError(f"indices must be [T, k] with 1 <= k <= {DISTILL_MAX_K}")
    _vector(indices, "indices", torch.int64, (T, k))
    _vector(logits, "logits", torch.float32, (T, k))
    if teacher_lse is not None:
        _vector(teacher_lse, "teacher_lse", torch.float32, (T,))
    return _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, stream, k,
                 lambda h, s: dgl_linear_distill(h, indices.data_ptr(), logits.data_ptr(),
                                                 teacher_lse.data_ptr() if teacher_lse is not None else None, k,
                                                 temperature, s), "dgl_linear_distill")
