"""ctypes declarations of libqmm.so (the C ABI in include/qmm.h).  Marshalling only."""
from __future__ import annotations

import ctypes
import os

QMM_MAX_DIMS = 8
QMM_DECODE_MAX_ROWS = 32
QMM_BF16 = 1
QMM_FP16 = 2
QMM_FLAG_FORCE_STRIDED = 1

ERRORS = {
    0: "QMM_OK",
    -1: "QMM_ERR_NULL",
    -2: "QMM_ERR_UNSUPPORTED",
    -3: "QMM_ERR_SHAPE",
    -4: "QMM_ERR_LAYOUT",
    -5: "QMM_ERR_ALIGN",
    -6: "QMM_ERR_HIP",
}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmm.so")

# Every symbol include/qmm.h declares.
EXPORTS = ("qmm_abi_version", "qmm_last_error", "qmm_quantize", "qmv", "qmm_t", "qmm_plan", "qmm_gather_qmv",
           "qmm_dequantize", "qmm_embedding", "qmm_qmv_argmax", "qmm_qmv_argmax_noalloc", "qmm_topk",
           "qmm_qmv_topk", "qmm_kv_append", "qmm_kv_read", "qmm_kv_attend", "qmm_kv_attend_workspace_bytes", "qmm_sample", "qmm_moe",
           "qmm_moe_workspace_bytes")


class TensorDesc(ctypes.Structure):
    _fields_ = [("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * QMM_MAX_DIMS),
                ("stride", ctypes.c_int64 * QMM_MAX_DIMS)]


class WeightDesc(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p),
                ("w_row_stride", ctypes.c_int64),
                ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p),
                ("sb_row_stride", ctypes.c_int64),
                ("N", ctypes.c_int64),
                ("K", ctypes.c_int64),
                ("group_size", ctypes.c_int32),
                ("bits", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64),
                ("batches", ctypes.c_int64),
                ("batch_stride", ctypes.c_int64),
                ("rows_per_batch", ctypes.c_int64),
                ("seg_rows", ctypes.c_int64),
                ("seg_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64),
                ("family", ctypes.c_int32),
                ("kind", ctypes.c_int32)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p),
                ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class KVAttendDesc(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p),
                ("q_batch_stride", ctypes.c_int64),
                ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64),
                ("batch", ctypes.c_int64),
                ("q_len", ctypes.c_int64),
                ("q_heads", ctypes.c_int32),
                ("causal", ctypes.c_int32),
                ("window", ctypes.c_int64),
                ("scale", ctypes.c_float),
                ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64),
                ("max_blocks", ctypes.c_int64),
                ("lengths", ctypes.c_void_p),
                ("max_length", ctypes.c_int64)]


class ExpertStack(ctypes.Structure):
    _fields_ = [("w", WeightDesc),
                ("num_experts", ctypes.c_int64),
                ("w_expert_stride", ctypes.c_int64),
                ("sb_expert_stride", ctypes.c_int64)]


class MoeDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64),
                ("router_logits", ctypes.c_void_p),
                ("router_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int64),
                ("top_k", ctypes.c_int32),
                ("renormalize", ctypes.c_int32),
                ("dtype", ctypes.c_int32),
                ("gate", ctypes.POINTER(ExpertStack)),
                ("up", ctypes.POINTER(ExpertStack)),
                ("down", ctypes.POINTER(ExpertStack)),
                ("y_stride", ctypes.c_int64)]


class SampleParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p),
                ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p),
                ("temperature_all", ctypes.c_float),
                ("top_k_all", ctypes.c_int32),
                ("top_p_all", ctypes.c_float),
                ("min_p_all", ctypes.c_float)]


class QmmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__("%s (%d): %s" % (ERRORS.get(code, "?"), code, message))
        self.code = code
        self.message = message


_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree libqmm.so; fail loudly when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libqmm.so is not built (%s); run `python -m bit_affine_quantized_qmv_amd.build`"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    lib.qmm_abi_version.restype = ctypes.c_int32
    lib.qmm_abi_version.argtypes = []
    lib.qmm_last_error.restype = ctypes.c_char_p
    lib.qmm_last_error.argtypes = []
    lib.qmm_quantize.restype = ctypes.c_int32
    lib.qmm_quantize.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                 ctypes.c_int32, ctypes.c_int32, P, P, P, P]
    for name in ("qmv", "qmm_t"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int32
        fn.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc), P,
                       ctypes.POINTER(TensorDesc), ctypes.c_uint32, P]
    lib.qmm_gather_qmv.restype = ctypes.c_int32
    lib.qmm_gather_qmv.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc), ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int64, P, P, ctypes.POINTER(TensorDesc), P]
    lib.qmm_qmv_argmax.restype = ctypes.c_int32
    lib.qmm_qmv_argmax.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc), P,
                                   ctypes.POINTER(TensorDesc), P, P, P, P]
    lib.qmm_qmv_argmax_noalloc.restype = ctypes.c_int32
    lib.qmm_qmv_argmax_noalloc.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc), P,
                                           ctypes.POINTER(TensorDesc), P, P, P]
    lib.qmm_topk.restype = ctypes.c_int32
    lib.qmm_topk.argtypes = [P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                             P, P, P, P]
    lib.qmm_qmv_topk.restype = ctypes.c_int32
    lib.qmm_qmv_topk.argtypes = [P, ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc), P,
                                 ctypes.POINTER(TensorDesc), ctypes.c_int32, P, P, P, P]
    lib.qmm_dequantize.restype = ctypes.c_int32
    lib.qmm_dequantize.argtypes = [ctypes.POINTER(WeightDesc), P, ctypes.c_int64, P]
    lib.qmm_embedding.restype = ctypes.c_int32
    lib.qmm_embedding.argtypes = [ctypes.POINTER(WeightDesc), P, ctypes.c_int64, P, ctypes.c_int64, P]
    lib.qmm_plan.restype = ctypes.c_int32
    lib.qmm_plan.argtypes = [ctypes.POINTER(TensorDesc), ctypes.POINTER(WeightDesc),
                             ctypes.POINTER(TensorDesc), ctypes.c_uint32, ctypes.c_int32,
                             ctypes.POINTER(Plan)]
    lib.qmm_kv_append.restype = ctypes.c_int32
    lib.qmm_kv_append.argtypes = [ctypes.POINTER(KVCacheDesc), P, ctypes.c_int64, ctypes.c_int64, P, ctypes.c_int64,
                                  ctypes.c_int64, P, ctypes.c_int64, P]
    lib.qmm_kv_read.restype = ctypes.c_int32
    lib.qmm_kv_read.argtypes = [ctypes.POINTER(KVCacheDesc), P, ctypes.c_int64, P, P, P]
    lib.qmm_kv_attend.restype = ctypes.c_int32
    lib.qmm_kv_attend.argtypes = [ctypes.POINTER(KVCacheDesc), ctypes.POINTER(KVAttendDesc), P, P, ctypes.c_int64, P]
    lib.qmm_kv_attend_workspace_bytes.restype = ctypes.c_int64
    lib.qmm_kv_attend_workspace_bytes.argtypes = [ctypes.POINTER(KVCacheDesc), ctypes.POINTER(KVAttendDesc)]
    lib.qmm_sample.restype = ctypes.c_int32
    lib.qmm_sample.argtypes = [P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                               ctypes.POINTER(SampleParams), P, P, P, P, P]
    lib.qmm_moe.restype = ctypes.c_int32
    lib.qmm_moe.argtypes = [ctypes.POINTER(MoeDesc), P, P, ctypes.c_int64, P]
    lib.qmm_moe_workspace_bytes.restype = ctypes.c_int64
    lib.qmm_moe_workspace_bytes.argtypes = [ctypes.c_int64] * 5
    _lib = lib
    return lib


def check(rc: int) -> None:
    if rc != 0:
        raise QmmError(rc, load().qmm_last_error().decode())


def tensor_desc(shape, stride) -> TensorDesc:
    d = TensorDesc()
    d.ndim = len(shape)
    for i, (s, st) in enumerate(zip(shape, stride)):
        d.shape[i] = int(s)
        d.stride[i] = int(st)
    return d
