"""Affine group-quantized matmul (qmv / qmm_t) on AMD MI355X (gfx950).

The computation lives in libqmm.so (hand-written HIP kernels behind the C ABI of
include/qmm.h); this package only marshals torch tensors into those calls.
"""
from ._lib import (QMM_BF16, QMM_DECODE_MAX_ROWS, QMM_FLAG_FORCE_STRIDED, QMM_FP16, QmmError,
                   load)
from .api import (ExpertWeights, QuantizedWeight, argmax_workspace, dequantize, embedding, gather_qmv, plan, qmm_t, qmv,
                  qmv_argmax, qmv_argmax_noalloc, qmv_topk, quantize, topk, topk_workspace)
from .kv import KVCache, kv_append, kv_attend, kv_attend_workspace, kv_cache, kv_read
from .experts import grouped_qmm, grouped_workspace, moe, moe_prompt, moe_prompt_workspace, moe_workspace
from .trees import (kv_attend_tree, kv_attend_tree_workspace, kv_copy_pages, kv_fork, kv_move, tree_accept, tree_mask)
from .sampling import sample, sample_workspace

__all__ = ["QMM_BF16", "QMM_FP16", "QMM_FLAG_FORCE_STRIDED", "QMM_DECODE_MAX_ROWS", "QmmError",
           "QuantizedWeight", "ExpertWeights", "argmax_workspace", "dequantize", "embedding", "gather_qmv", "qmv_argmax", "qmv_argmax_noalloc", "qmv_topk", "topk", "topk_workspace", "load", "plan", "qmm_t", "qmv", "quantize",
           "KVCache", "kv_cache", "kv_append", "kv_read", "kv_attend", "kv_attend_workspace", "moe", "moe_workspace", "sample",
           "sample_workspace", "tree_mask", "tree_accept", "kv_attend_tree", "kv_attend_tree_workspace", "kv_move",
           "kv_copy_pages", "kv_fork", "grouped_qmm", "grouped_workspace", "moe_prompt", "moe_prompt_workspace"]
