"""ctypes binding over libqgemv.so (the C ABI declared in include/qgemv.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their data pointers and the current HIP stream are passed to the
library, and a non-zero status raises ``QgError``.  Every computation runs in
the library's HIP kernels; there is no fallback of any kind.  PyTorch is used
for device memory (output and workspace allocation) and streams.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, fields
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemv.so")

QG_OK = 0
QG_ERR_DEVICE_CHECK = 7  # QG_DEBUG=1 (or 2) only: a device-side check of the outlier path failed
QG_F32, QG_BF16 = 0, 1
QG_INT8, QG_FP8 = 2, 3
QG_PER_TENSOR, QG_PER_ROW = 0, 1
QG_WFMT_INT8, QG_WFMT_TERNARY2, QG_WFMT_SIGN1_RES8, QG_WFMT_Q4K, QG_WFMT_SIGN1_RES8Z, QG_WFMT_TERNARY3 = 0, 1, 2, 3, 4, 5
QG_WFMT_INT8_T16 = 6
QG_WFMT_FP8, QG_WFMT_FP8_T16 = 7, 8
QG_ACT_INT8, QG_ACT_FLOAT = 0, 1
QG_MAX_OUTLIERS = 256
QG_QGEMV_MAX_K = 32768
QG_MAX_GROUP = 8
QG_OUT_LD_ALIGN = 8
QG_MAX_OUT_LD = 65536
QG_SEP_MAX_K = 65536
QG_BATCH_MAX_M = 16
QG_BATCH_MAX_K = 262144
QG_MX_BLOCK = 32
QG_QGEMM_MAX_K = 133120
QG_ABSMAX_SCRATCH_PARTS = 1024
QG_MAX_ROW_GROUPS = 1024
QG_MAX_PLAN_ROWS = 1 << 30
QG_MAX_TOP_K = 16
QG_LORA_MAX_R = 256
QG_FP8_BLOCK = 128
QG_ROW_MAX_K = 32768
QG_CHAIN_MAX_STAGES = 4096
QG_CHAIN_MIN_K = 128
QG_CHAIN_MAX_K = 16384
QG_CHAIN_ERROR_OFFSET = 64
QG_CHAIN_TIMEOUT_TICKS = 200000000

_c_i32, _c_i64, _c_sz, _c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class QgError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" % (what, status_str(status), status))
        self.status = status


class CWeight(ctypes.Structure):
    _fields_ = [("fmt", _c_i32), ("reserved", _c_i32), ("n", _c_i64), ("k", _c_i64),
                ("codes", _c_vp), ("resid", _c_vp), ("scale", _c_vp), ("scale2", _c_vp), ("zero", _c_vp)]


class CSepMatrix(ctypes.Structure):
    _fields_ = [("cls", _c_vp), ("rv", _c_vp), ("rv_ld", _c_i64), ("alpha", _c_vp), ("s_r", _c_vp), ("n", _c_i64),
                ("y", _c_vp), ("acc_out", _c_vp)]


class CChainStage(ctypes.Structure):
    _fields_ = [("count", _c_i32), ("dep", _c_i32), ("x", _c_vp), ("w", ctypes.POINTER(CWeight)),
                ("y", ctypes.POINTER(_c_vp))]


class CRowGroups(ctypes.Structure):
    _fields_ = [("offsets", _c_vp), ("order", _c_vp), ("rows", _c_i64), ("groups", _c_i32), ("per_row", _c_i32)]


class CExperts(ctypes.Structure):
    _fields_ = [("fmt", _c_i32), ("reserved", _c_i32), ("e", _c_i64), ("n", _c_i64), ("k", _c_i64),
                ("codes", _c_vp), ("scale", _c_vp)]


class CLora(ctypes.Structure):
    _fields_ = [("a", _c_vp), ("b", _c_vp), ("scale", _c_vp), ("n", _c_i64), ("r", _c_i32), ("reserved", _c_i32),
                ("y", _c_vp)]


_SIGS = {
    "qg_status_str": (ctypes.c_char_p, [_c_i32]),
    "qg_abi_version": (_c_i32, []),
    "qg_quantize_absmax_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i32]),
    "qg_quantize_absmax": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_quantize_absmax_noalloc": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp, _c_vp]),
    "qg_probe_stream_read_bytes": (_c_sz, [_c_i64, _c_i32]),
    "qg_probe_stream_read": (_c_i32, [_c_vp, _c_i64, _c_i32, _c_vp, _c_vp]),
    "qg_chain_plan_bytes": (_c_sz, [ctypes.POINTER(CChainStage), _c_i32, _c_i32]),
    "qg_chain_plan": (_c_i32, [ctypes.POINTER(CChainStage), _c_i32, _c_i32, _c_vp, _c_sz]),
    "qg_qgemv_chain": (_c_i32, [_c_vp, _c_vp, _c_vp]),
    "qg_quantize_absmax_split": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i32, _c_vp, _c_vp, _c_vp, _c_i32,
                                          _c_vp]),
    "qg_detect_outliers_workspace_bytes": (_c_sz, [_c_i64]),
    "qg_detect_outliers": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_gather_columns_bf16": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i32, _c_vp, _c_i32, _c_vp]),
    "qg_ternary_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "qg_quantize_ternary": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_split_sign_residual": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "qg_split_sign_residual_zp": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "qg_quantize_asym": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp]),
    "qg_quantize_q4k": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "qg_qgemv_batch": (_c_i32, [ctypes.POINTER(CWeight), _c_i32, _c_vp, _c_i32, _c_vp, _c_i32, _c_vp]),
    "qg_qgemv_batch_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i32]),
    "qg_qgemv_batch_ws": (_c_i32, [ctypes.POINTER(CWeight), _c_i32, _c_vp, _c_i32, _c_vp, _c_i32, _c_vp, _c_sz, _c_vp]),
    "qg_qgemv_batch_grouped": (_c_i32, [ctypes.POINTER(CWeight), _c_i32, _c_i32, _c_vp, _c_i32,
                                        ctypes.POINTER(_c_vp), _c_i32, _c_vp]),
    "qg_quantize_mxfp4": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "qg_gemm_mxfp4": (_c_i32, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "qg_prefill_mxfp4_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "qg_prefill_mxfp4": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_sep_resid_ld": (_c_i64, [_c_i64, _c_i32]),
    "qg_split_sep_threshold": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_i32, _c_i32, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp,
                                        _c_vp]),
    "qg_qgemv_sep": (_c_i32, [_c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_i32, _c_i32, _c_vp,
                              _c_vp, _c_vp]),
    "qg_qgemv_sep_grouped": (_c_i32, [ctypes.POINTER(CSepMatrix), _c_i32, _c_i64, _c_vp, _c_i32, _c_i32, _c_vp]),
    "qg_pack": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp]),
    "qg_base3_row_bytes": (_c_i64, [_c_i64]),
    "qg_pack_base3": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "qg_tiles16_bytes": (_c_i64, [_c_i64, _c_i64]),
    "qg_pack_tiles16": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "qg_unpack_base3": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "qg_unpack": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp]),
    "qg_qgemv": (_c_i32, [ctypes.POINTER(CWeight), _c_i32, _c_vp, _c_i32, _c_vp, _c_i32, _c_vp, _c_vp]),
    "qg_qgemv_grouped": (_c_i32, [ctypes.POINTER(CWeight), _c_i32, _c_i32, _c_vp, _c_i32, ctypes.POINTER(_c_vp),
                                  _c_i32, ctypes.POINTER(_c_vp), _c_vp]),
    "qg_qgemm_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i32]),
    "qg_qgemm_w8a8_outlier": (_c_i32, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i32, _c_vp, _c_vp, _c_vp, _c_i32, _c_i64,
                                       _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_group_rows_workspace_bytes": (_c_sz, [_c_i64, _c_i32]),
    "qg_group_rows": (_c_i32, [_c_vp, _c_i64, _c_i32, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "qg_moe_route": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i32, _c_i32, _c_i32, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                              _c_sz, _c_vp]),
    "qg_qgemm_experts": (_c_i32, [ctypes.POINTER(CExperts), ctypes.POINTER(CRowGroups), _c_i32, _c_vp, _c_vp, _c_i64,
                                  _c_vp, _c_i32, _c_vp]),
    "qg_qgemm_experts_swiglu": (_c_i32, [ctypes.POINTER(CExperts), ctypes.POINTER(CExperts),
                                         ctypes.POINTER(CRowGroups), _c_i32, _c_vp, _c_vp, _c_i64, _c_vp, _c_i32,
                                         _c_vp]),
    "qg_experts_combine_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "qg_qgemm_experts_combine": (_c_i32, [ctypes.POINTER(CExperts), ctypes.POINTER(CRowGroups), _c_i32, _c_vp, _c_vp,
                                          _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i32, _c_vp, _c_sz, _c_vp]),
    "qg_lora_workspace_bytes": (_c_sz, [ctypes.POINTER(CLora), _c_i32, _c_i64, _c_i32, _c_i64]),
    "qg_lora_add": (_c_i32, [ctypes.POINTER(CLora), _c_i32, ctypes.POINTER(CRowGroups), _c_vp, _c_i64, _c_i64, _c_i32,
                             _c_vp, _c_sz, _c_vp]),
    "qg_quantize_fp8": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "qg_quantize_fp8_weight": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "qg_rms_norm": (_c_i32, [_c_vp, _c_i32, _c_vp, _c_vp, _c_vp, _c_i32, ctypes.c_float, _c_i64, _c_i64, _c_i32, _c_vp,
                             _c_vp, _c_vp]),
    "qg_swiglu": (_c_i32, [_c_vp, _c_i32, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp, _c_vp]),
    "qg_qgemm_fp8_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32]),
    "qg_qgemm_fp8": (_c_i32, [ctypes.POINTER(CWeight), _c_vp, _c_vp, _c_i64, _c_vp, _c_i32, _c_vp, _c_sz, _c_vp]),
    "qg_qgemm_w8a8": (_c_i32, [_c_vp, _c_vp, _c_vp, _c_i32, _c_i64, _c_i64, _c_i32, _c_vp, _c_vp, _c_vp, _c_i32,
                               _c_i64, _c_vp, _c_vp, _c_vp]),
}
EXPORTED = tuple(_SIGS)

_lib = None


def lib() -> ctypes.CDLL:
    """Load libqgemv.so (built in-tree by quantized_gemv_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libqgemv.so is not built (%s); run quantized_gemv_amd.build.build()" % LIB_PATH)
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def status_str(st: int) -> str:
    return lib().qg_status_str(st).decode()


def _check(st: int, what: str):
    if st != QG_OK:
        raise QgError(st, what)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    return t


def _xt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return QG_F32
    if t.dtype == torch.bfloat16:
        return QG_BF16
    raise ValueError("activation dtype must be float32 or bfloat16")


def _idx_host(idx: Optional[Sequence[int]]):
    if idx is None:
        return None, 0
    arr = (ctypes.c_int32 * max(len(idx), 1))(*[int(v) for v in idx])
    return arr, len(idx)


# ------------------------------------------------------------------ quantizers

def quantize_absmax(x: torch.Tensor, per_row: bool = True, q: torch.Tensor = None, s: torch.Tensor = None):
    """Symmetric absmax int8 quantization (qg_quantize_absmax). Returns (q, s)."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    rows, cols = (1, x.shape[0]) if x.dim() == 1 else tuple(x.shape)
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device) if q is None else _dev(q, "q", torch.int8)
    s = torch.empty(rows if per_row else 1, dtype=torch.float32, device=x.device) if s is None else _dev(s, "s", torch.float32)
    gran = QG_PER_ROW if per_row else QG_PER_TENSOR
    nws = lib().qg_quantize_absmax_workspace_bytes(rows, cols, gran)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=x.device) if nws else None
    _check(lib().qg_quantize_absmax(_p(x), _xt(x), rows, cols, gran, _p(q), _p(s), _p(ws), nws, _stream(x)),
           "qg_quantize_absmax")
    return q, s


def out_ld(n_out: int) -> int:
    """Row stride of an outlier operand the prefill GEMMs read: n_out rounded
    up to QG_OUT_LD_ALIGN elements."""
    return -(-n_out // QG_OUT_LD_ALIGN) * QG_OUT_LD_ALIGN


def quantize_absmax_split(x: torch.Tensor, idx: Sequence[int], ld: Optional[int] = None):
    """Per-token int8 quantization with outlier channels split out
    (qg_quantize_absmax_split). Returns (q, s, x_out) with x_out [rows][ld]
    (ld defaults to out_ld(n_out); columns >= n_out are zero)."""
    _dev(x, "x", torch.bfloat16)
    rows, cols = x.shape
    cidx, n_out = _idx_host(idx)
    ld = out_ld(n_out) if ld is None else ld
    q = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    s = torch.empty(rows, dtype=torch.float32, device=x.device)
    xo = torch.empty((rows, ld), dtype=torch.bfloat16, device=x.device)
    _check(lib().qg_quantize_absmax_split(_p(x), rows, cols, cidx, n_out, _p(q), _p(s), _p(xo) if n_out else None,
                                          ld, _stream(x)), "qg_quantize_absmax_split")
    return q, s, xo


def detect_outliers(x: torch.Tensor, n_out: int, ws: torch.Tensor = None) -> torch.Tensor:
    """The n_out channels of calibration activations x [rows][cols] (bf16)
    with the largest max |x| (qg_detect_outliers). Returns int32 [n_out] on
    the device, ascending."""
    _dev(x, "x", torch.bfloat16)
    rows, cols = x.shape
    idx = torch.empty(n_out, dtype=torch.int32, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, lib().qg_detect_outliers_workspace_bytes(cols)), dtype=torch.uint8, device=x.device)
    _check(lib().qg_detect_outliers(_p(x), rows, cols, n_out, _p(idx) if n_out else None, _p(ws), ws.numel(),
                                    _stream(x)), "qg_detect_outliers")
    return idx


def gather_columns_bf16(w: torch.Tensor, idx: Sequence[int], ld: Optional[int] = None):
    """W_out[n][j] = bf16(W[n][idx[j]]) (qg_gather_columns_bf16), as [n][ld]
    (ld defaults to out_ld(n_out); columns >= n_out are zero)."""
    _dev(w, "w", torch.float32)
    n, k = w.shape
    cidx, n_out = _idx_host(idx)
    ld = out_ld(n_out) if ld is None else ld
    wo = torch.empty((n, ld), dtype=torch.bfloat16, device=w.device)
    _check(lib().qg_gather_columns_bf16(_p(w), n, k, cidx, n_out, _p(wo) if n_out else None, ld, _stream(w)),
           "qg_gather_columns_bf16")
    return wo


def quantize_ternary(w: torch.Tensor):
    """Ternary absmean quantization (qg_quantize_ternary). Returns (codes, gamma[1])."""
    _dev(w, "w", torch.float32)
    n, k = (1, w.shape[0]) if w.dim() == 1 else tuple(w.shape)
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    g = torch.empty(1, dtype=torch.float32, device=w.device)
    nws = lib().qg_ternary_workspace_bytes(n, k)
    ws = torch.empty(nws, dtype=torch.uint8, device=w.device)
    _check(lib().qg_quantize_ternary(_p(w), n, k, _p(q), _p(g), _p(ws), nws, _stream(w)), "qg_quantize_ternary")
    return q, g


def split_sign_residual(w: torch.Tensor):
    """Sign backbone + int8 residual split (qg_split_sign_residual).
    Returns (sign int8, alpha, rq int8, s_r)."""
    _dev(w, "w", torch.float32)
    n, k = w.shape
    sign = torch.empty((n, k), dtype=torch.int8, device=w.device)
    rq = torch.empty((n, k), dtype=torch.int8, device=w.device)
    alpha = torch.empty(n, dtype=torch.float32, device=w.device)
    s_r = torch.empty(n, dtype=torch.float32, device=w.device)
    _check(lib().qg_split_sign_residual(_p(w), n, k, _p(sign), _p(alpha), _p(rq), _p(s_r), _stream(w)),
           "qg_split_sign_residual")
    return sign, alpha, rq, s_r


def split_sign_residual_zp(w: torch.Tensor):
    """Sign backbone + asymmetric int8 residual (qg_split_sign_residual_zp).
    Returns (sign int8, alpha, rq int8, s_r, z_r int8)."""
    _dev(w, "w", torch.float32)
    n, k = w.shape
    sign = torch.empty((n, k), dtype=torch.int8, device=w.device)
    rq = torch.empty((n, k), dtype=torch.int8, device=w.device)
    alpha = torch.empty(n, dtype=torch.float32, device=w.device)
    s_r = torch.empty(n, dtype=torch.float32, device=w.device)
    z_r = torch.empty(n, dtype=torch.int8, device=w.device)
    _check(lib().qg_split_sign_residual_zp(_p(w), n, k, _p(sign), _p(alpha), _p(rq), _p(s_r), _p(z_r), _stream(w)),
           "qg_split_sign_residual_zp")
    return sign, alpha, rq, s_r, z_r


def quantize_asym(x: torch.Tensor):
    """Asymmetric int8 quantization per row (qg_quantize_asym): x [rows][cols]
    fp32 or bf16. Returns (q int8, s fp32 [rows], z int8 [rows])."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if x.dim() != 2:
        raise ValueError("x must be [rows][cols]")
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    s = torch.empty(rows, dtype=torch.float32, device=x.device)
    z = torch.empty(rows, dtype=torch.int8, device=x.device)
    _check(lib().qg_quantize_asym(_p(x), _xt(x), rows, cols, _p(q), _p(s), _p(z), _stream(x)), "qg_quantize_asym")
    return q, s, z


def pack(codes: torch.Tensor, bits: int, out: torch.Tensor = None):
    """Bit packing (qg_pack): bits=2 ternary, bits=1 sign."""
    _dev(codes, "codes", torch.int8)
    n, k = (1, codes.shape[0]) if codes.dim() == 1 else tuple(codes.shape)
    if bits not in (1, 2) or k % (8 // bits):
        raise ValueError("bad bits or row length")
    out = torch.empty((n, k * bits // 8), dtype=torch.uint8, device=codes.device) if out is None else out
    _check(lib().qg_pack(_p(codes), n, k, bits, _p(out), _stream(codes)), "qg_pack")
    return out


def unpack(packed: torch.Tensor, bits: int, k: int):
    """Inverse of pack (qg_unpack)."""
    _dev(packed, "packed", torch.uint8)
    n = packed.shape[0] if packed.dim() == 2 else 1
    out = torch.empty((n, k), dtype=torch.int8, device=packed.device)
    _check(lib().qg_unpack(_p(packed), n, k, bits, _p(out), _stream(packed)), "qg_unpack")
    return out


def base3_row_bytes(k: int) -> int:
    """Bytes of one base-3 packed row (qg_base3_row_bytes): 16 per 80 weights."""
    return int(lib().qg_base3_row_bytes(k))


def pack_base3(codes: torch.Tensor, out: torch.Tensor = None):
    """Ternary codes, five per byte (qg_pack_base3): [n][k] int8 -> [n][base3_row_bytes(k)] uint8."""
    _dev(codes, "codes", torch.int8)
    n, k = (1, codes.shape[0]) if codes.dim() == 1 else tuple(codes.shape)
    rb = base3_row_bytes(k)
    out = torch.empty((n, rb), dtype=torch.uint8, device=codes.device) if out is None else out
    _check(lib().qg_pack_base3(_p(codes), n, k, _p(out), _stream(codes)), "qg_pack_base3")
    return out


def pack_tiles16(codes: torch.Tensor, out: torch.Tensor = None):
    """Int8 codes [n][k] in 16-row tiles for the batch products
    (qg_pack_tiles16): returns a flat int8 tensor of qg_tiles16_bytes(n, k)."""
    _dev(codes, "codes", torch.int8)
    if codes.dim() != 2:
        raise ValueError("codes must be [n][k]")
    n, k = codes.shape
    nb = int(lib().qg_tiles16_bytes(n, k))
    if nb == 0:
        raise ValueError("shape (%d, %d) has no 16-row tiled layout" % (n, k))
    out = torch.empty(nb, dtype=torch.int8, device=codes.device) if out is None else out
    if out.numel() < nb:
        raise ValueError("out holds %d bytes, %d needed" % (out.numel(), nb))
    _call("qg_pack_tiles16", codes, codes.data_ptr(), n, k, out.data_ptr())
    return out


def tiled16(w: "QWeight") -> "QWeight":
    """The QG_WFMT_INT8 (or QG_WFMT_FP8) matrix w with its codes in 16-row tiles."""
    if w.fmt == QG_WFMT_FP8:
        t = pack_tiles16(w.codes.view(torch.int8).view(w.n, w.k))
        return QWeight(QG_WFMT_FP8_T16, w.n, w.k, t.view(w.codes.dtype), w.scale)
    if w.fmt != QG_WFMT_INT8:
        raise ValueError("tiled16 takes QG_WFMT_INT8 or QG_WFMT_FP8 weights")
    return QWeight(QG_WFMT_INT8_T16, w.n, w.k, pack_tiles16(w.codes.view(w.n, w.k)), w.scale)


def unpack_base3(packed: torch.Tensor, k: int):
    """Inverse of pack_base3 (qg_unpack_base3)."""
    _dev(packed, "packed", torch.uint8)
    n = packed.shape[0] if packed.dim() == 2 else 1
    out = torch.empty((n, k), dtype=torch.int8, device=packed.device)
    _check(lib().qg_unpack_base3(_p(packed), n, k, _p(out), _stream(packed)), "qg_unpack_base3")
    return out


# ------------------------------------------------------------------ products

@dataclass
class QWeight:
    """A quantized weight matrix as the library stores it."""
    fmt: int
    n: int
    k: int
    codes: torch.Tensor
    scale: Optional[torch.Tensor]
    resid: Optional[torch.Tensor] = None
    scale2: Optional[torch.Tensor] = None
    zero: Optional[torch.Tensor] = None

    def c_struct(self) -> CWeight:
        return CWeight(self.fmt, 0, self.n, self.k, self.codes.data_ptr(),
                       self.resid.data_ptr() if self.resid is not None else None,
                       self.scale.data_ptr() if self.scale is not None else None,
                       self.scale2.data_ptr() if self.scale2 is not None else None,
                       self.zero.data_ptr() if self.zero is not None else None)


def quantize_q4k(w: torch.Tensor):
    """Group-wise 4-bit codes with two-level scales (qg_quantize_q4k).
    Returns (codes plane uint8 [n][k/2], meta plane uint8 [n][k/256][16]);
    QWeight(QG_WFMT_Q4K, n, k, codes, None, resid=meta) describes them."""
    _dev(w, "w", torch.float32)
    n, k = w.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    meta = torch.empty((n, k // 256, 16), dtype=torch.uint8, device=w.device)
    _check(lib().qg_quantize_q4k(_p(w), n, k, _p(codes), _p(meta), _stream(w)), "qg_quantize_q4k")
    return codes, meta


def qgemv_batch(w: QWeight, x: torch.Tensor, y_dtype=torch.float32, y: torch.Tensor = None,
                ws: Optional[torch.Tensor] = None):
    """Weight-only int8 product of a batch of tokens (qg_qgemv_batch): x bf16
    [m][k] -> y [m][n]. Returns y.  With ws (a uint8 device tensor of at least
    batch_workspace_bytes(w.n, w.k, m) bytes, zero-filled when allocated) the
    call is qg_qgemv_batch_ws (K split over workgroups)."""
    _dev(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be [m][k]")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, w.n), dtype=y_dtype, device=x.device)
    _dev(y, "y", (torch.float32, torch.bfloat16))
    cw = w.c_struct()
    if ws is None:
        _check(lib().qg_qgemv_batch(ctypes.byref(cw), m, _p(x), QG_BF16, _p(y), _xt(y), _stream(x)), "qg_qgemv_batch")
    else:
        _dev(ws, "ws", torch.uint8)
        _check(lib().qg_qgemv_batch_ws(ctypes.byref(cw), m, _p(x), QG_BF16, _p(y), _xt(y), _p(ws), ws.numel(),
                                       _stream(x)), "qg_qgemv_batch_ws")
    return y


def batch_workspace_bytes(n: int, k: int, m: int) -> int:
    """Workspace of qg_qgemv_batch_ws (0: the split path does not apply)."""
    return int(lib().qg_qgemv_batch_workspace_bytes(n, k, m))


def qgemv_batch_grouped(weights: Sequence[QWeight], x: torch.Tensor, y_dtype=torch.float32, ys=None):
    """qg_qgemv_batch_grouped: several int8 matrices sharing x [m][k] in one
    launch. Returns the list of y [m][n_j]."""
    _dev(x, "x", torch.bfloat16)
    m = x.shape[0]
    cnt = len(weights)
    if not 1 <= cnt <= QG_MAX_GROUP:
        raise ValueError("need 1..%d weights" % QG_MAX_GROUP)
    if ys is None:
        ys = [torch.empty((m, W.n), dtype=y_dtype, device=x.device) for W in weights]
    arr = (CWeight * cnt)(*[W.c_struct() for W in weights])
    yp = (_c_vp * cnt)(*[y.data_ptr() for y in ys])
    _check(lib().qg_qgemv_batch_grouped(arr, cnt, m, _p(x), QG_BF16, yp, _xt(ys[0]), _stream(x)),
           "qg_qgemv_batch_grouped")
    return ys


def quantize_mxfp4(x: torch.Tensor):
    """MXFP4 quantization of the rows of x [rows][cols] (fp32 or bf16)
    (qg_quantize_mxfp4). Returns (codes uint8 [rows][cols/2], scales uint8
    [cols/256][rows][8])."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    r, c = x.shape
    codes = torch.empty((r, c // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((c // 256, r, 8), dtype=torch.uint8, device=x.device)
    _check(lib().qg_quantize_mxfp4(_p(x), _xt(x), r, c, _p(codes), _p(scales), _stream(x)), "qg_quantize_mxfp4")
    return codes, scales


def gemm_mxfp4(a, a_scales, b, b_scales, y: torch.Tensor = None):
    """Y = A B^T of two MXFP4 operands (qg_gemm_mxfp4). Returns y fp32 [m][n]."""
    for t, nm in ((a, "a"), (a_scales, "a_scales"), (b, "b"), (b_scales, "b_scales")):
        _dev(t, nm, torch.uint8)
    m, n, k = a.shape[0], b.shape[0], 2 * a.shape[1]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=a.device)
    _dev(y, "y", torch.float32)
    _check(lib().qg_gemm_mxfp4(_p(a), _p(a_scales), m, k, _p(b), _p(b_scales), n, _p(y), _stream(a)),
           "qg_gemm_mxfp4")
    return y


def prefill_mxfp4(x: torch.Tensor, w, w_scales, y: torch.Tensor = None, ws: torch.Tensor = None):
    """Format-separated prefill (qg_prefill_mxfp4): x bf16 [m][k] quantized to
    MXFP4 in the workspace, times the MXFP4 weights. Returns y fp32 [m][n]."""
    _dev(x, "x", torch.bfloat16)
    m, k = x.shape
    n = w.shape[0]
    need = int(lib().qg_prefill_mxfp4_workspace_bytes(m, k))
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check(lib().qg_prefill_mxfp4(_p(x), m, k, _p(w), _p(w_scales), n, _p(y), _p(ws), ws.numel(), _stream(x)),
           "qg_prefill_mxfp4")
    return y


class SepWeight:
    """Thresholded separated weights as qg_split_sep_threshold writes them:
    cls [n][k/4] uint8 (2-bit classes), rv [n][ld] int8 (residual codes in
    increasing k, then zeros), alpha [n] and s_r [n] fp32."""

    def __init__(self, cls: torch.Tensor, rv: torch.Tensor, alpha: torch.Tensor, s_r: torch.Tensor, k: int):
        self.cls, self.rv, self.alpha, self.s_r = cls, rv, alpha, s_r
        self.n, self.k = cls.shape[0], k
        self.ld = rv.shape[1]


def sep_resid_ld(k: int, pct_zero: int) -> int:
    """Smallest valid row stride of the residual stream (qg_sep_resid_ld)."""
    return int(lib().qg_sep_resid_ld(k, pct_zero))


def split_sep_threshold(w: torch.Tensor, pct_backbone: int = 80, pct_zero: int = 50, ld: Optional[int] = None):
    """Thresholded separated split (qg_split_sep_threshold). Returns SepWeight."""
    _dev(w, "w", torch.float32)
    n, k = w.shape
    if ld is None:
        ld = sep_resid_ld(k, pct_zero)
    cls = torch.empty((n, k // 4), dtype=torch.uint8, device=w.device)
    rv = torch.empty((n, max(int(ld), 1)), dtype=torch.int8, device=w.device)
    alpha = torch.empty(n, dtype=torch.float32, device=w.device)
    s_r = torch.empty(n, dtype=torch.float32, device=w.device)
    _check(lib().qg_split_sep_threshold(_p(w), n, k, pct_backbone, pct_zero, _p(cls), _p(rv), int(ld), _p(alpha),
                                        _p(s_r), _stream(w)), "qg_split_sep_threshold")
    return SepWeight(cls, rv, alpha, s_r, k)


def qgemv_sep(sw: SepWeight, x: torch.Tensor, skip_residual: bool = False, y: torch.Tensor = None,
              acc_out: torch.Tensor = None):
    """Batch-1 product on thresholded separated weights (qg_qgemv_sep);
    acc_out, if given, is int32 [2][n] (backbone, residual). Returns y (fp32)."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if y is None:
        y = torch.empty(sw.n, dtype=torch.float32, device=x.device)
    _dev(y, "y", torch.float32)
    if acc_out is not None:
        _dev(acc_out, "acc_out", torch.int32)
    _check(lib().qg_qgemv_sep(_p(sw.cls), _p(sw.rv), sw.ld, _p(sw.alpha), _p(sw.s_r), sw.n, sw.k, _p(x), _xt(x),
                              1 if skip_residual else 0, _p(y), _p(acc_out), _stream(x)), "qg_qgemv_sep")
    return y


class SepGroupLaunch:
    """Pre-marshalled arguments of one qg_qgemv_sep_grouped call: products of
    1..QG_MAX_GROUP thresholded separated matrices on the same x (kept alive
    by this object); launch() enqueues it on x's current stream."""

    def __init__(self, weights: Sequence[SepWeight], x: torch.Tensor, ys: Sequence[torch.Tensor],
                 skip_residual: bool = False, accs: Optional[Sequence[torch.Tensor]] = None):
        _dev(x, "x", (torch.float32, torch.bfloat16))
        n = len(weights)
        if not 1 <= n <= QG_MAX_GROUP or len(ys) != n or (accs is not None and len(accs) != n):
            raise ValueError("need 1..%d weights and as many outputs" % QG_MAX_GROUP)
        for y in ys:
            _dev(y, "y", torch.float32)
        if accs is not None:
            for a in accs:
                if a is not None:
                    _dev(a, "acc_out", torch.int32)
        self.keep = (list(weights), x, list(ys), accs)
        self.m = (CSepMatrix * n)(*[
            CSepMatrix(_p(w.cls), _p(w.rv), w.ld, _p(w.alpha), _p(w.s_r), w.n, _p(y),
                       None if accs is None or accs[i] is None else _p(accs[i]))
            for i, (w, y) in enumerate(zip(weights, ys))])
        self.n, self.k, self.x, self.xt = n, weights[0].k, x, _xt(x)
        self.skip = 1 if skip_residual else 0

    def launch(self):
        _check(lib().qg_qgemv_sep_grouped(self.m, self.n, self.k, _p(self.x), self.xt, self.skip, _stream(self.x)),
               "qg_qgemv_sep_grouped")


def qgemv_sep_grouped(weights: Sequence[SepWeight], x: torch.Tensor, skip_residual: bool = False,
                      accs: Optional[Sequence[torch.Tensor]] = None):
    """Thresholded separated products on the same x in one launch
    (qg_qgemv_sep_grouped). Returns [y] (fp32)."""
    ys = [torch.empty(w.n, dtype=torch.float32, device=x.device) for w in weights]
    SepGroupLaunch(weights, x, ys, skip_residual, accs).launch()
    return ys


def qgemv(w: QWeight, x: torch.Tensor, act_int8: bool, y_dtype=torch.float32, y: torch.Tensor = None,
          acc_out: torch.Tensor = None):
    """Batch-1 quantized GEMV (qg_qgemv). Returns y."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    if y is None:
        y = torch.empty(w.n, dtype=y_dtype, device=x.device)
    _dev(y, "y", (torch.float32, torch.bfloat16))
    if acc_out is not None:
        _dev(acc_out, "acc_out", torch.int32)
    cw = w.c_struct()
    _check(lib().qg_qgemv(ctypes.byref(cw), QG_ACT_INT8 if act_int8 else QG_ACT_FLOAT, _p(x), _xt(x), _p(y), _xt(y),
                          _p(acc_out), _stream(x)), "qg_qgemv")
    return y


class GroupLaunch:
    """Pre-marshalled arguments of one qg_qgemv_grouped call (kept alive by
    this object); launch() enqueues it on the current stream."""

    def __init__(self, weights: Sequence[QWeight], x: torch.Tensor, ys: Sequence[torch.Tensor], act_int8: bool,
                 accs: Optional[Sequence[torch.Tensor]] = None):
        _dev(x, "x", (torch.float32, torch.bfloat16))
        n = len(weights)
        if not 1 <= n <= QG_MAX_GROUP or len(ys) != n:
            raise ValueError("need 1..%d weights and as many outputs" % QG_MAX_GROUP)
        for y in ys:
            _dev(y, "y", (torch.float32, torch.bfloat16))
        self.x, self.ys, self.accs = x, list(ys), accs
        self.cw = (CWeight * n)(*[w.c_struct() for w in weights])
        self.yp = (_c_vp * n)(*[y.data_ptr() for y in ys])
        self.ap = None if accs is None else (_c_vp * n)(*[None if a is None else a.data_ptr() for a in accs])
        self.n = n
        self.amode = QG_ACT_INT8 if act_int8 else QG_ACT_FLOAT
        self.xt = _xt(x)
        self.yt = _xt(ys[0])

    def launch(self):
        _check(lib().qg_qgemv_grouped(self.cw, self.n, self.amode, _p(self.x), self.xt, self.yp, self.yt, self.ap,
                                      _stream(self.x)), "qg_qgemv_grouped")


def qgemv_grouped(weights: Sequence[QWeight], x: torch.Tensor, act_int8: bool, y_dtype=torch.float32,
                  accs: Optional[Sequence[torch.Tensor]] = None):
    """Several GEMVs on the same x in one launch (qg_qgemv_grouped). Returns [y]."""
    ys = [torch.empty(w.n, dtype=y_dtype, device=x.device) for w in weights]
    GroupLaunch(weights, x, ys, act_int8, accs).launch()
    return ys


def qgemv_launch_raw(cw: CWeight, amode: int, x_ptr: int, xt: int, y_ptr: int, yt: int, stream_ptr: int) -> int:
    """Pre-marshalled launch for tight timing loops (returns the status)."""
    return lib().qg_qgemv(ctypes.byref(cw), amode, ctypes.c_void_p(x_ptr), xt, ctypes.c_void_p(y_ptr), yt, None,
                          ctypes.c_void_p(stream_ptr))


def qgemm_w8a8_outlier(x: torch.Tensor, idx: Sequence[int], wq: torch.Tensor, s_w: torch.Tensor,
                       w_out: Optional[torch.Tensor], y: torch.Tensor = None, acc_out: torch.Tensor = None,
                       ws: torch.Tensor = None):
    """W8A8 prefill GEMM with the outlier split (qg_qgemm_w8a8_outlier). Returns y."""
    _dev(x, "x", torch.bfloat16)
    _dev(wq, "wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    m, k = x.shape
    n = wq.shape[0]
    cidx, n_out = _idx_host(idx)
    w_ld = 0
    if n_out:
        _dev(w_out, "w_out", torch.bfloat16)
        w_ld = w_out.shape[1]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    nws = lib().qg_qgemm_workspace_bytes(m, k, n_out)
    if ws is None:
        ws = torch.empty(nws, dtype=torch.uint8, device=x.device)
    _check(lib().qg_qgemm_w8a8_outlier(_p(x), m, k, cidx, n_out, _p(wq), _p(s_w), _p(w_out) if n_out else None, w_ld,
                                       n, _p(y), _p(acc_out), _p(ws), ws.numel(), _stream(x)), "qg_qgemm_w8a8_outlier")
    return y


def qgemm_w8a8(xq: torch.Tensor, s_x: torch.Tensor, x_out: Optional[torch.Tensor], wq: torch.Tensor,
               s_w: torch.Tensor, w_out: Optional[torch.Tensor], n_out: int, y: torch.Tensor = None,
               acc_out: torch.Tensor = None):
    """The GEMM half of the prefill on already split activations (qg_qgemm_w8a8):
    xq [m][k] int8, s_x [m], x_out [m][x_ld] bf16 and w_out [n][w_ld] bf16 (as
    quantize_absmax_split / gather_columns_bf16 return them), n_out outlier
    channels. Returns y [m][n] fp32."""
    _dev(xq, "xq", torch.int8)
    _dev(s_x, "s_x", torch.float32)
    _dev(wq, "wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    m, k = xq.shape
    n = wq.shape[0]
    x_ld = w_ld = 0
    if n_out:
        _dev(x_out, "x_out", torch.bfloat16)
        _dev(w_out, "w_out", torch.bfloat16)
        x_ld, w_ld = x_out.shape[1], w_out.shape[1]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=xq.device)
    _check(lib().qg_qgemm_w8a8(_p(xq), _p(s_x), _p(x_out) if n_out else None, x_ld, m, k, n_out, _p(wq), _p(s_w),
                               _p(w_out) if n_out else None, w_ld, n, _p(y), _p(acc_out), _stream(xq)),
           "qg_qgemm_w8a8")
    return y


# ------------------------------------------------------------------ products whose matrix depends on the row

def _same_device(x: torch.Tensor, *others: Optional[torch.Tensor]):
    index = x.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors are on %s and %s" % (x.device, t.device))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent in builds without a GPU backend


def _call(name: str, x: torch.Tensor, *args):
    """The entry point `name` on x's current stream (appended as the last
    argument), with x's device current for the launch."""
    index = x.get_device()
    f = getattr(_lib or lib(), name)
    if index == torch._C._cuda_getDevice():
        st = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = f(*args, _raw_stream(index))
    if st != QG_OK:
        raise QgError(st, name)


def _shaped(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor):
    """t, checked, or a new tensor of that shape and dtype on like's device."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    _same_device(like, t)
    return t


def _workspace(ws: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """(tensor or None, bytes) of a workspace of at least `need` bytes."""
    if ws is None:
        return (torch.empty(need, dtype=torch.uint8, device=like.device), need) if need else (None, 0)
    _dev(ws, "ws", torch.uint8)
    _same_device(like, ws)
    return ws, ws.numel()


def _memory(*tensors: Optional[torch.Tensor]):
    """What keeps the tensors' memory where it is, also if their data is set
    anew (a module that moves does that to its parameters)."""
    return [t.untyped_storage() for t in tensors if t is not None]


class _FromFields:
    """Copied, saved and loaded by its fields: the addresses that an object
    holds are those of its own tensors."""

    def __reduce__(self):
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


@dataclass(frozen=True)
class RowGroups(_FromFields):
    """A row plan (qg_group_rows): the rows sorted by group. offsets
    [groups + 1], order and pos [rows], int32 on the device; per_row plan rows
    read one row of x (a router's top_k).  Checked once, when it is made: calls
    read and write the memory that the tensors have then."""
    offsets: torch.Tensor
    order: torch.Tensor
    pos: torch.Tensor
    per_row: int = 1

    def __post_init__(self):
        for t, nm in ((self.offsets, "offsets"), (self.order, "order"), (self.pos, "pos")):
            _dev(t, nm, torch.int32)
        _same_device(self.offsets, self.order, self.pos)
        if self.order.numel() != self.pos.numel():
            raise ValueError("order and pos differ in length")
        put = object.__setattr__
        put(self, "groups", self.offsets.numel() - 1)
        put(self, "rows", self.order.numel())
        put(self, "ptrs", (self.offsets.data_ptr(), self.order.data_ptr(), self.pos.data_ptr()))
        put(self, "_keep", _memory(self.offsets, self.order, self.pos))
        put(self, "_c", tuple(CRowGroups(self.ptrs[0], order, self.rows, self.groups, self.per_row)
                              for order in (None, self.ptrs[1])))

    def c_struct(self, gather: bool = True) -> CRowGroups:
        return self._c[1 if gather else 0]


@dataclass(frozen=True)
class Routing(_FromFields):
    """What moe_route returns: ids and weights [tokens][top_k] and the plan.
    Checked once, when it is made."""
    ids: torch.Tensor
    weights: torch.Tensor
    groups: RowGroups

    def __post_init__(self):
        _dev(self.ids, "ids", torch.int32)
        _dev(self.weights, "weights", torch.float32)
        _same_device(self.ids, self.weights, self.groups.offsets)
        if self.ids.dim() != 2 or self.weights.shape != self.ids.shape or self.ids.numel() != self.groups.rows \
                or self.ids.shape[1] != self.groups.per_row:
            raise ValueError("ids and weights must be [tokens][top_k], one per row of the plan")
        object.__setattr__(self, "_keep", _memory(self.ids, self.weights))
        object.__setattr__(self, "ptrs", (self.ids.data_ptr(), self.weights.data_ptr()) + self.groups.ptrs)


def _plan_buffers(x: torch.Tensor, rows: int, groups: int, per_row: int, out: Optional[RowGroups]) -> RowGroups:
    if out is None:
        i32 = dict(dtype=torch.int32, device=x.device)
        return RowGroups(torch.empty(groups + 1, **i32), torch.empty(rows, **i32), torch.empty(rows, **i32), per_row)
    if out.rows != rows or out.groups != groups or out.per_row != per_row:
        raise ValueError("out holds %d rows of %d groups, per_row %d; %d, %d, %d needed"
                         % (out.rows, out.groups, out.per_row, rows, groups, per_row))
    _same_device(x, out.offsets)
    return out


def group_rows(ids: torch.Tensor, groups: int, out: Optional[RowGroups] = None,
               ws: Optional[torch.Tensor] = None) -> RowGroups:
    """Rows sorted by id (qg_group_rows): ids int32 [rows], or [tokens][top_k]
    as another router gives them (per_row = top_k); ids outside [0, groups)
    have no group. -> RowGroups.  A serving step makes one plan of its rows'
    adapters and uses it for every layer and projection."""
    _dev(ids, "ids", torch.int32)
    if ids.dim() not in (1, 2):
        raise ValueError("ids must be [rows] or [tokens][top_k]")
    rows = ids.numel()
    out = _plan_buffers(ids, rows, groups, 1 if ids.dim() == 1 else ids.shape[1], out)
    ws, nws = _workspace(ws, int(lib().qg_group_rows_workspace_bytes(rows, groups)), ids)
    _call("qg_group_rows", ids, _ptr(ids), rows, groups, *out.ptrs, _ptr(ws), nws)
    return out


def moe_route(logits: torch.Tensor, top_k: int, renorm: bool = True, out: Optional[Routing] = None,
              ws: Optional[torch.Tensor] = None) -> Routing:
    """Top-k router and the plan of its choice (qg_moe_route): logits
    [tokens][experts] fp32 or bf16 -> Routing."""
    _dev(logits, "logits", (torch.float32, torch.bfloat16))
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens][experts]")
    t, e = logits.shape
    if out is None:
        out = Routing(torch.empty((t, top_k), dtype=torch.int32, device=logits.device),
                      torch.empty((t, top_k), dtype=torch.float32, device=logits.device),
                      _plan_buffers(logits, t * top_k, e, top_k, None))
    else:
        _plan_buffers(logits, t * top_k, e, top_k, out.groups)
    ws, nws = _workspace(ws, int(lib().qg_group_rows_workspace_bytes(t * top_k, e)), logits)
    _call("qg_moe_route", logits, logits.data_ptr(), _xt(logits), t, e, top_k, 1 if renorm else 0, *out.ptrs, _ptr(ws),
          nws)
    return out


@dataclass(frozen=True)
class QExperts(_FromFields):
    """The experts' int8 matrices (qg_experts): codes [e][n][k] (QG_WFMT_INT8)
    or each expert's 16-row tiles (QG_WFMT_INT8_T16, tiled16_experts), scale
    [e][n]."""
    fmt: int
    e: int
    n: int
    k: int
    codes: torch.Tensor
    scale: torch.Tensor

    def __post_init__(self):
        _dev(self.codes, "codes", torch.int8)
        _dev(self.scale, "scale", torch.float32)
        _same_device(self.codes, self.scale)
        per = (self.n + 15) // 16 * 16 if self.fmt == QG_WFMT_INT8_T16 else self.n
        if self.codes.numel() != self.e * per * self.k or self.scale.numel() != self.e * self.n:
            raise ValueError("codes or scale do not hold %d experts of [%d][%d]" % (self.e, self.n, self.k))
        at = (self.codes.data_ptr(), self.scale.data_ptr())
        object.__setattr__(self, "_at", at)
        object.__setattr__(self, "_c", CExperts(self.fmt, 0, self.e, self.n, self.k, *at))

    def c_struct(self) -> CExperts:
        # weights whose data was set anew (a module moved) are not where they were
        if (self.codes.data_ptr(), self.scale.data_ptr()) != self._at:
            self.__post_init__()
        return self._c


def quantize_experts(w: torch.Tensor) -> QExperts:
    """Per-row absmax int8 (qg_quantize_absmax) of the experts' matrices
    w [e][n][k] (fp32 or bf16)."""
    if w.dim() != 3:
        raise ValueError("w must be [e][n][k]")
    e, n, k = w.shape
    with torch.cuda.device(w.device):
        q, s = quantize_absmax(w.view(e * n, k), per_row=True)
    return QExperts(QG_WFMT_INT8, e, n, k, q.view(e, n, k), s.view(e, n))


def tiled16_experts(w: QExperts) -> QExperts:
    """The QG_WFMT_INT8 experts w with each one's codes in 16-row tiles (one
    qg_pack_tiles16 per expert; done once, when the weights are loaded)."""
    if w.fmt != QG_WFMT_INT8:
        raise ValueError("tiled16_experts takes QG_WFMT_INT8 experts")
    nb = int(lib().qg_tiles16_bytes(w.n, w.k))
    if nb == 0:
        raise ValueError("shape (%d, %d) has no 16-row tiled layout" % (w.n, w.k))
    out = torch.empty((w.e, nb), dtype=torch.int8, device=w.codes.device)
    codes = w.codes.view(w.e, w.n, w.k)
    with torch.cuda.device(codes.device):
        for j in range(w.e):
            pack_tiles16(codes[j], out[j])
    return QExperts(QG_WFMT_INT8_T16, w.e, w.n, w.k, out, w.scale)


def _experts_x(w: QExperts, x: torch.Tensor, groups: RowGroups, s_x: Optional[torch.Tensor], gather: bool) -> int:
    """Checks x (bf16, or int8 codes with s_x) against w and the plan; the
    activation mode."""
    _dev(x, "x", (torch.bfloat16, torch.int8))
    if x.dim() != 2 or x.shape[1] != w.k:
        raise ValueError("x must be [rows][%d]" % w.k)
    if (x.dtype == torch.int8) != (s_x is not None):
        raise ValueError("int8 x needs s_x, bf16 x takes none")
    if s_x is not None:
        _dev(s_x, "s_x", torch.float32)
        if s_x.numel() != x.shape[0]:
            raise ValueError("s_x must hold one scale per row of x")
    if groups.per_row < 1:
        raise ValueError("the plan's per_row is %d" % groups.per_row)
    want = -(-groups.rows // groups.per_row) if gather else groups.rows
    if x.shape[0] != want:
        raise ValueError("x has %d rows, the plan reads %d" % (x.shape[0], want))
    if groups.groups != w.e:
        raise ValueError("the plan has %d groups for %d experts" % (groups.groups, w.e))
    _same_device(x, w.codes, s_x, groups.offsets)
    return QG_ACT_FLOAT if s_x is None else QG_ACT_INT8


def _y_dtype(y: Optional[torch.Tensor], y_dtype):
    dt = y_dtype if y is None else y.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("y is float32 or bfloat16")
    return dt


def qgemm_experts(w: QExperts, x: torch.Tensor, groups: RowGroups, s_x: Optional[torch.Tensor] = None,
                  gather: bool = True, y_dtype=torch.float32, y: torch.Tensor = None) -> torch.Tensor:
    """Products grouped by expert (qg_qgemm_experts): x bf16 [x_rows][k]
    (W8A16), or int8 codes with s_x [x_rows] (W8A8). Returns y [rows][n] in the
    plan's order; rows behind the last group are not written. gather=False: x
    is in the plan's order already."""
    amode = _experts_x(w, x, groups, s_x, gather)
    y = _shaped(y, "y", (groups.rows, w.n), _y_dtype(y, y_dtype), x)
    cg = groups.c_struct(gather)
    _call("qg_qgemm_experts", x, ctypes.byref(w.c_struct()), ctypes.byref(cg), amode, _ptr(x), _ptr(s_x), x.shape[0], _ptr(y),
          _xt(y))
    return y


def qgemm_experts_swiglu(gate: QExperts, up: QExperts, x: torch.Tensor, groups: RowGroups,
                         s_x: Optional[torch.Tensor] = None, gather: bool = True, y_dtype=torch.bfloat16,
                         y: torch.Tensor = None) -> torch.Tensor:
    """silu(gate product) * up product, grouped by expert, in one launch
    (qg_qgemm_experts_swiglu). Returns y [rows][n] in the plan's order."""
    amode = _experts_x(gate, x, groups, s_x, gather)
    _same_device(x, up.codes)
    y = _shaped(y, "y", (groups.rows, gate.n), _y_dtype(y, y_dtype), x)
    cg = groups.c_struct(gather)
    _call("qg_qgemm_experts_swiglu", x, ctypes.byref(gate.c_struct()), ctypes.byref(up.c_struct()), ctypes.byref(cg),
          amode, _ptr(x), _ptr(s_x), x.shape[0], _ptr(y), _xt(y))
    return y


def qgemm_experts_combine(w: QExperts, x: torch.Tensor, groups: RowGroups, weights: torch.Tensor,
                          s_x: Optional[torch.Tensor] = None, gather: bool = False, y_dtype=torch.float32,
                          y: torch.Tensor = None, ws: torch.Tensor = None) -> torch.Tensor:
    """Products grouped by expert, added per token with the router's weights
    [tokens][top_k] (qg_qgemm_experts_combine). x is in the plan's order (the
    output of qgemm_experts_swiglu) unless gather. Returns y [tokens][n]."""
    amode = _experts_x(w, x, groups, s_x, gather)
    _dev(weights, "weights", torch.float32)
    tokens = groups.rows // groups.per_row
    if weights.numel() != groups.rows or tokens * groups.per_row != groups.rows:
        raise ValueError("weights must be [tokens][%d], one per row of the plan" % groups.per_row)
    _same_device(x, weights)
    y = _shaped(y, "y", (tokens, w.n), _y_dtype(y, y_dtype), x)
    ws, nws = _workspace(ws, int(lib().qg_experts_combine_workspace_bytes(groups.rows, w.n)), x)
    cg = groups.c_struct(gather)
    _call("qg_qgemm_experts_combine", x, ctypes.byref(w.c_struct()), ctypes.byref(cg), amode, _ptr(x), _ptr(s_x), x.shape[0],
          groups.ptrs[2], _ptr(weights), tokens, _ptr(y), _xt(y), _ptr(ws), nws)
    return y


def moe_ffn(x: torch.Tensor, logits: torch.Tensor, gate: QExperts, up: QExperts, down: QExperts, top_k: int,
            renorm: bool = True, act_int8: bool = False, y_dtype=torch.bfloat16) -> torch.Tensor:
    """The expert feed-forward of x bf16 [tokens][k]: moe_route of the
    router's logits, SwiGLU of the gate and up products, the down product
    combined per token. act_int8: both products W8A8, their activations
    quantized per row (quantize_absmax). Returns y [tokens][down.n]."""
    r = moe_route(logits, top_k, renorm)
    s_x = s_h = None
    if act_int8:
        with torch.cuda.device(x.device):
            x, s_x = quantize_absmax(x, per_row=True)
    h = qgemm_experts_swiglu(gate, up, x, r.groups, s_x=s_x)
    if act_int8:
        with torch.cuda.device(h.device):
            h, s_h = quantize_absmax(h, per_row=True)
    return qgemm_experts_combine(down, h, r.groups, r.weights, s_x=s_h, y_dtype=y_dtype)


@dataclass
class LoraAdapters:
    """Low-rank adapters of one projection: a [groups][r][k] and b
    [groups][n][r] bf16, scale fp32 [groups] or None (1). Fields may be set
    anew: they are checked when the object is made and by every LoraLaunch."""
    a: torch.Tensor
    b: torch.Tensor
    scale: Optional[torch.Tensor] = None

    def __post_init__(self):
        self.check()

    def check(self):
        """ValueError unless the fields, as they are now, fit together."""
        _dev(self.a, "a", torch.bfloat16)
        _dev(self.b, "b", torch.bfloat16)
        if self.a.dim() != 3 or self.b.dim() != 3 or self.a.shape[0] != self.b.shape[0] or self.a.shape[1] != self.b.shape[2]:
            raise ValueError("a must be [groups][r][k] and b [groups][n][r]")
        if self.scale is not None:
            _dev(self.scale, "scale", torch.float32)
            if self.scale.numel() != self.a.shape[0]:
                raise ValueError("scale must be [groups]")
        _same_device(self.a, self.b, self.scale)


class LoraLaunch:
    """Pre-marshalled arguments of one qg_lora_add call: the adapters of
    1..QG_MAX_GROUP projections of the same x, as they are now, added to ys
    (all kept alive by this object, with a workspace); launch() enqueues it on
    x's current stream. Launches that may overlap need objects of their own:
    they share ys and the workspace. The object may be dropped while launches
    run, on any stream: its own workspace waits for them. The tensors given to it
    follow torch's rule (on a stream other than the one they were made on, they
    are kept or recorded by the caller). While a graph that captured a launch may
    be replayed, the object has to be kept."""

    def __init__(self, x: torch.Tensor, groups: RowGroups, adapters: Sequence[LoraAdapters],
                 ys: Sequence[torch.Tensor], ws: Optional[torch.Tensor] = None):
        _dev(x, "x", torch.bfloat16)
        n = len(adapters)
        if not 1 <= n <= QG_MAX_GROUP or len(ys) != n:
            raise ValueError("need 1..%d adapters and as many outputs" % QG_MAX_GROUP)
        if x.dim() != 2 or x.shape[0] != groups.rows:
            raise ValueError("x must be [%d][k], a row per row of the plan" % groups.rows)
        _same_device(x, groups.offsets)
        m, k = x.shape
        for ad, y in zip(adapters, ys):
            _dev(y, "y", (torch.float32, torch.bfloat16))
            LoraAdapters.check(ad)  # its fields may have been set anew
            _same_device(x, ad.a, y)
            if ad.a.shape[0] != groups.groups or ad.a.shape[2] != k:
                raise ValueError("a must be [%d][r][%d]" % (groups.groups, k))
            if tuple(y.shape) != (m, ad.b.shape[1]) or y.dtype != ys[0].dtype:
                raise ValueError("each y must be [%d][n] of its b, all of one dtype" % m)
        self.m = (CLora * n)(*[
            CLora(ad.a.data_ptr(), ad.b.data_ptr(), None if ad.scale is None else ad.scale.data_ptr(), ad.b.shape[1],
                  ad.a.shape[1], 0, y.data_ptr()) for ad, y in zip(adapters, ys)])
        self.ws, self.nws = _workspace(ws, int(lib().qg_lora_workspace_bytes(self.m, n, m, groups.groups, k)), x)
        # the stream that a workspace of this object's own comes from
        self.made_on = None if self.ws is ws else _raw_stream(x.get_device())
        self.cg = groups.c_struct()
        self.ys = list(ys)
        # the memory itself: adapters whose fields, or tensors whose data, are set
        # anew later do not take it away from these arguments
        self.x, self.index = x.detach(), x.get_device()
        self.keep = (groups, _memory(x, self.ws, *ys, *(t for ad in adapters for t in (ad.a, ad.b, ad.scale))))
        # as C values: converted once, not by every launch
        self.args = (ctypes.cast(self.m, ctypes.POINTER(CLora)), _c_i32(n), ctypes.pointer(self.cg), _c_vp(x.data_ptr()),
                     _c_i64(m), _c_i64(k), _c_i32(_xt(ys[0])), _c_vp(_ptr(self.ws)), _c_sz(self.nws))

    def launch(self):
        for y in self.ys:
            if y.requires_grad and torch.is_grad_enabled():
                raise ValueError("adapters are added in place, without a gradient: a y requires one")
        if self.made_on is not None and _raw_stream(self.index) != self.made_on:
            # no one else knows of this use: once dropped, the workspace would go
            # to the next tensor of its own stream while the kernels still run
            self.ws.record_stream(torch.cuda.current_stream(self.x.device))
        _call("qg_lora_add", self.x, *self.args)
        # a backward pass that has saved a y must see that it changed
        torch._C._increment_version(self.ys)


def lora_add(x: torch.Tensor, groups: RowGroups, adapters: Sequence[LoraAdapters], ys: Sequence[torch.Tensor],
             ws: Optional[torch.Tensor] = None):
    """Adds the rows' low-rank adapters (qg_lora_add) to the projections' outputs
    ys [rows][n], in place: x bf16 [rows][k], groups = group_rows of the rows'
    adapter numbers (rows without one are left as they were). No gradient passes:
    a y that requires one is refused while gradients are on. Returns ys."""
    LoraLaunch(x, groups, adapters, ys, ws).launch()
    return ys


# ------------------------------------------------------------------ the 8-bit path between layers

_OUT = {torch.float32: QG_F32, torch.bfloat16: QG_BF16, torch.int8: QG_INT8, torch.float8_e4m3fn: QG_FP8}


def _rows_cols(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError("%s must be [rows][columns]" % name)
    return t.shape


def _out_dtype(y: Optional[torch.Tensor], dtype):
    dt = dtype if y is None else y.dtype
    if dt not in _OUT:
        raise ValueError("outputs are float32, bfloat16, int8 or float8_e4m3fn")
    return dt


def _scale_out(s: Optional[torch.Tensor], dt, rows: int, cols: int, x: torch.Tensor):
    """The scales of an 8-bit output (None for the others)."""
    if dt not in (torch.int8, torch.float8_e4m3fn):
        if s is not None:
            raise ValueError("float outputs have no scales")
        return None
    return _shaped(s, "s", (rows,) if dt == torch.int8 else (cols // QG_FP8_BLOCK, rows), torch.float32, x)


class _Launch:
    """Pre-marshalled arguments of one call, with its outputs: launch() enqueues
    it on x's current stream, again and again on the same memory. Launches that
    may overlap need objects of their own: they share the outputs and the
    workspace. The object may be dropped while launches run, on any stream: a
    workspace of its own waits for them. The tensors given to it, and its
    outputs, follow torch's rule (on a stream other than the one they were made
    on, they are kept or recorded by the caller). While a graph that captured a
    launch may be replayed, the object has to be kept. No gradient passes."""

    def _set(self, name: str, x: torch.Tensor, args, tensors, outs, own_ws: Optional[torch.Tensor] = None):
        # x for its device; the memory itself, also if tensors' data is set anew
        self._name, self._x = name, x.detach()
        # a workspace of this object's own, and the stream that it comes from
        self._ws, self._made_on = own_ws, None if own_ws is None else _raw_stream(x.get_device())
        self._args, self._keep = args, _memory(*tensors)
        self._outs = [t for t in outs if t is not None]

    def launch(self):
        for t in self._outs:
            if t.requires_grad and torch.is_grad_enabled():
                raise ValueError("outputs are written without a gradient: one requires a gradient")
        if self._ws is not None and _raw_stream(self._x.get_device()) != self._made_on:
            # no one else knows of this use: once dropped, it would go to the next
            # tensor of its own stream while the kernels still run
            self._ws.record_stream(torch.cuda.current_stream(self._x.device))
        _call(self._name, self._x, *self._args)
        # a backward pass that has saved an output must see that it changed
        torch._C._increment_version(self._outs)


class RmsNormLaunch(_Launch):
    """One qg_rms_norm call: x [rows][k] (fp32 or bf16), weight [k]; with a
    residual (x's shape and type) its sum goes to residual_out (residual itself
    by default). out_dtype, or y's: float32, bfloat16, int8 (s: a multiplier per
    row) or float8_e4m3fn (s [k/128][rows]). Fields y, s, residual_out hold the
    outputs."""

    def __init__(self, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, y: torch.Tensor = None,
                 s: torch.Tensor = None):
        _dev(x, "x", (torch.float32, torch.bfloat16))
        rows, k = _rows_cols(x, "x")
        _dev(weight, "weight", (torch.float32, torch.bfloat16))
        if weight.shape != (k,):
            raise ValueError("weight must be [%d]" % k)
        _same_device(x, weight)
        if residual is not None:
            residual = _shaped(residual, "residual", x.shape, x.dtype, x)
            residual_out = _shaped(residual if residual_out is None else residual_out, "residual_out", x.shape, x.dtype, x)
        elif residual_out is not None:
            raise ValueError("residual_out without a residual")
        dt = _out_dtype(y, out_dtype)
        self.y, self.residual_out = _shaped(y, "y", (rows, k), dt, x), residual_out
        self.s = _scale_out(s, dt, rows, k, x)
        args = (_c_vp(_ptr(x)), _c_i32(_xt(x)), _c_vp(_ptr(residual)), _c_vp(_ptr(residual_out)), _c_vp(_ptr(weight)),
                _c_i32(_xt(weight)), ctypes.c_float(eps), _c_i64(rows), _c_i64(k), _c_i32(_OUT[dt]), _c_vp(_ptr(self.y)),
                _c_vp(_ptr(self.s)))
        self._set("qg_rms_norm", x, args, (x, residual, weight, residual_out, self.y, self.s),
                  (self.y, self.s, residual_out))


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, y: torch.Tensor = None,
             s: torch.Tensor = None):
    """Root-mean-square norm of the rows of x, or of x + residual
    (qg_rms_norm, arguments as RmsNormLaunch); the sum replaces the residual
    unless residual_out is given. Returns y, or (y, s) of 8-bit outputs."""
    a = RmsNormLaunch(x, weight, eps, residual, residual_out, out_dtype, y, s)
    a.launch()
    return a.y if a.s is None else (a.y, a.s)


class SwigluLaunch(_Launch):
    """One qg_swiglu call: x [rows][2 n] (fp32 or bf16), gate's columns then
    up's. out_dtype (or y's), y and s as RmsNormLaunch."""

    def __init__(self, x: torch.Tensor, out_dtype=torch.bfloat16, y: torch.Tensor = None, s: torch.Tensor = None):
        _dev(x, "x", (torch.float32, torch.bfloat16))
        rows, n2 = _rows_cols(x, "x")
        if n2 % 2:
            raise ValueError("x must hold gate's and up's columns")
        n, dt = n2 // 2, _out_dtype(y, out_dtype)
        self.y = _shaped(y, "y", (rows, n), dt, x)
        self.s = _scale_out(s, dt, rows, n, x)
        args = (_c_vp(_ptr(x)), _c_i32(_xt(x)), _c_i64(rows), _c_i64(n), _c_i32(_OUT[dt]), _c_vp(_ptr(self.y)),
                _c_vp(_ptr(self.s)))
        self._set("qg_swiglu", x, args, (x, self.y, self.s), (self.y, self.s))


def swiglu(x: torch.Tensor, out_dtype=torch.bfloat16, y: torch.Tensor = None, s: torch.Tensor = None):
    """silu(gate) * up of x [rows][2 n] (qg_swiglu, arguments as SwigluLaunch).
    Returns y [rows][n], or (y, s) of 8-bit outputs."""
    a = SwigluLaunch(x, out_dtype, y, s)
    a.launch()
    return a.y if a.s is None else (a.y, a.s)


def quantize_fp8(x: torch.Tensor, q: torch.Tensor = None, s: torch.Tensor = None):
    """e4m3 codes of the rows of x [rows][cols] (fp32 or bf16), a step per 128
    columns (qg_quantize_fp8). Returns (q float8_e4m3fn, s [cols/128][rows])."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    rows, cols = _rows_cols(x, "x")
    given = [t for t in (q, s) if t is not None]
    if given and torch.is_grad_enabled() and any(t.requires_grad for t in given):
        raise ValueError("outputs are written without a gradient: one requires a gradient")
    # torch.empty_like and sizes that are no tuple take half the host time
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn) if q is None else _shaped(q, "q", x.shape, torch.float8_e4m3fn, x)
    if s is None:
        s = torch.empty(cols // QG_FP8_BLOCK, rows, dtype=torch.float32, device=x.device)
    else:
        _shaped(s, "s", (cols // QG_FP8_BLOCK, rows), torch.float32, x)
    _call("qg_quantize_fp8", x, x.data_ptr(), _xt(x), rows, cols, q.data_ptr(), s.data_ptr())
    if given:
        torch._C._increment_version(given)
    return q, s


def quantize_fp8_weight(w: torch.Tensor) -> QWeight:
    """e4m3 codes of w [n][k] (fp32 or bf16), a step per block of 128 x 128
    (qg_quantize_fp8_weight), as QG_WFMT_FP8. tiled16 lays them out in tiles."""
    _dev(w, "w", (torch.float32, torch.bfloat16))
    n, k = _rows_cols(w, "w")
    codes = torch.empty_like(w, dtype=torch.float8_e4m3fn)
    scale = torch.empty(-(-n // QG_FP8_BLOCK), k // QG_FP8_BLOCK, dtype=torch.float32, device=w.device)
    _call("qg_quantize_fp8_weight", w, w.data_ptr(), _xt(w), n, k, codes.data_ptr(), scale.data_ptr())
    return QWeight(QG_WFMT_FP8, n, k, codes, scale)


def _check_fp8_weight(w: QWeight):
    if w.fmt not in (QG_WFMT_FP8, QG_WFMT_FP8_T16):
        raise ValueError("weights must be QG_WFMT_FP8 or QG_WFMT_FP8_T16")
    _dev(w.codes, "codes", (torch.float8_e4m3fn, torch.uint8, torch.int8))
    _dev(w.scale, "scale", torch.float32)
    _same_device(w.codes, w.scale)
    n = -(-w.n // 16) * 16 if w.fmt == QG_WFMT_FP8_T16 else w.n
    if w.codes.numel() != n * w.k or w.scale.numel() != -(-w.n // QG_FP8_BLOCK) * (w.k // QG_FP8_BLOCK):
        raise ValueError("codes or scale do not hold a matrix of [%d][%d]" % (w.n, w.k))
    if w.scale.dim() > 1 and w.scale.shape != (-(-w.n // QG_FP8_BLOCK), w.k // QG_FP8_BLOCK):
        raise ValueError("scale must be [n/128][k/128]")


class QgemmFp8Launch(_Launch):
    """One qg_qgemm_fp8 call: w (QG_WFMT_FP8 or QG_WFMT_FP8_T16), x
    float8_e4m3fn [m][k] with its steps s_x [k/128][m]; the output is y [m][n]
    (fp32 or bf16). ws: uint8, qg_qgemm_fp8_workspace_bytes, or the object's own."""

    def __init__(self, w: QWeight, x: torch.Tensor, s_x: torch.Tensor, y_dtype=torch.bfloat16, y: torch.Tensor = None,
                 ws: Optional[torch.Tensor] = None):
        _check_fp8_weight(w)
        _dev(x, "x", torch.float8_e4m3fn)
        m, k = _rows_cols(x, "x")
        if k != w.k:
            raise ValueError("x must be [m][%d]" % w.k)
        _dev(s_x, "s_x", torch.float32)
        if s_x.shape != (k // QG_FP8_BLOCK, m):
            raise ValueError("s_x must be [%d][%d]" % (k // QG_FP8_BLOCK, m))
        _same_device(x, s_x, w.codes)
        self.y = _shaped(y, "y", (m, w.n), _y_dtype(y, y_dtype), x)
        self._w = w.c_struct()
        need = int(lib().qg_qgemm_fp8_workspace_bytes(m, w.n, k, _xt(self.y)))
        ws_t, nws = _workspace(ws, need, x)
        args = (ctypes.pointer(self._w), _c_vp(_ptr(x)), _c_vp(_ptr(s_x)), _c_i64(m), _c_vp(_ptr(self.y)),
                _c_i32(_xt(self.y)), _c_vp(_ptr(ws_t)), _c_sz(nws))
        self._set("qg_qgemm_fp8", x, args, (x, s_x, w.codes, w.scale, self.y, ws_t), (self.y,),
                  ws_t if ws is None else None)


def qgemm_fp8(w: QWeight, x: torch.Tensor, s_x: torch.Tensor, y_dtype=torch.bfloat16, y: torch.Tensor = None,
              ws: Optional[torch.Tensor] = None):
    """Product of e4m3 operands in blocks of 128 (qg_qgemm_fp8, arguments as
    QgemmFp8Launch), from one token to prefill. Returns y [m][n]."""
    a = QgemmFp8Launch(w, x, s_x, y_dtype, y, ws)
    a.launch()
    return a.y


def fp8_ffn(x: torch.Tensor, residual: torch.Tensor, norm_weight: torch.Tensor, gate_up: QWeight, down: QWeight,
            eps: float = 1e-6) -> torch.Tensor:
    """A feed-forward layer on e4m3 weights: norm of x + residual (which becomes
    the residual), gate and up in one product (their matrices one after the
    other: [2 n][k]), SwiGLU, the way down. x bf16 [tokens][k]; returns bf16
    [tokens][down.n], to be added to the residual by the next norm."""
    q, s = rms_norm(x, norm_weight, eps, residual, out_dtype=torch.float8_e4m3fn)
    h, s_h = swiglu(qgemm_fp8(gate_up, q, s), out_dtype=torch.float8_e4m3fn)
    return qgemm_fp8(down, h, s_h)


def chain_plan_image(stages, workgroups: int):
    """qg_chain_plan on the host: `stages` is a list of (CWeight array, count,
    x pointer, y pointer array, dep).  Returns the 16-B aligned uint8 image
    (a numpy view) and the status; nothing is sent to a device."""
    import numpy as np
    n = len(stages)
    cs = (CChainStage * n)()
    for i, (cw, count, x_ptr, yp, dep) in enumerate(stages):
        cs[i].count, cs[i].dep, cs[i].x = count, dep, x_ptr
        cs[i].w = ctypes.cast(cw, ctypes.POINTER(CWeight))
        cs[i].y = ctypes.cast(yp, ctypes.POINTER(_c_vp))
    nbytes = lib().qg_chain_plan_bytes(cs, n, workgroups)
    raw = np.zeros(max(int(nbytes), 64) + 16, np.uint8)
    off = (-raw.ctypes.data) % 16
    img = raw[off:off + max(int(nbytes), 64)]
    st = lib().qg_chain_plan(cs, n, workgroups, ctypes.c_void_p(img.ctypes.data), nbytes)
    return img, st


class ChainStep:
    """The weight-only int8 products of a decode step with their data
    dependencies, run as one launch (qg_chain_plan once, then qg_qgemv_chain
    per call).

    stages: list of (weights, x, ys, dep): weights a list of QG_WFMT_INT8
    QWeights sharing k, x a bf16 tensor [k], ys bf16 tensors [n] (one per
    weight), dep the index of the stage whose outputs x holds (-1: none)."""

    def __init__(self, stages, workgroups: Optional[int] = None):
        self.keep = []
        plan = []
        dev = None
        for weights, x, ys, dep in stages:
            _dev(x, "x", torch.bfloat16)
            dev = x.device
            for y in ys:
                _dev(y, "y", torch.bfloat16)
            cw = (CWeight * len(weights))(*[w.c_struct() for w in weights])
            yp = (_c_vp * len(ys))(*[y.data_ptr() for y in ys])
            self.keep += [cw, yp, x, list(ys), list(weights)]
            plan.append((cw, len(weights), x.data_ptr(), yp, dep))
        if workgroups is None:
            workgroups = torch.cuda.get_device_properties(dev).multi_processor_count
        self.image, st = chain_plan_image(plan, workgroups)
        _check(st, "qg_chain_plan")
        self.plan = torch.from_numpy(self.image.copy()).to(dev)
        self.device = dev

    def launch(self):
        _check(lib().qg_qgemv_chain(ctypes.c_void_p(self.image.ctypes.data), _p(self.plan), _stream(self.plan)),
               "qg_qgemv_chain")

    def error(self) -> int:
        """The plan's error word (nonzero: a wait ran past its time bound)."""
        return int(self.plan[QG_CHAIN_ERROR_OFFSET:QG_CHAIN_ERROR_OFFSET + 4].view(torch.int32).item())

    def restore(self):
        """Copy the plan image to the device again (after an error)."""
        self.plan.copy_(torch.from_numpy(self.image))
