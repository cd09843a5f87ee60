"""The mixture-of-experts layer for a few tokens (qmm_moe).  Argument marshalling only, like
api.py."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _DTYPE_CODE, ExpertWeights
from .kv import raw_stream, same_device


def _stack(w: ExpertWeights) -> _lib.ExpertStack:
    codes, scales, biases = w.w_packed, w.scales, w.biases
    ce, cr, cl = codes.stride()
    se, sr, sl = scales.stride()
    assert cl == 1 and sl == 1 and (se, sr, sl) == biases.stride() and codes.dtype == torch.int32
    return _lib.ExpertStack(_lib.WeightDesc(codes.data_ptr(), cr, scales.data_ptr(), biases.data_ptr(), sr, w.N, w.K,
                                            w.group_size, w.bits, _DTYPE_CODE[scales.dtype]),
                            codes.size(0), ce, se)


def _bytes(lib, tokens: int, gate: ExpertWeights, top_k: int) -> int:
    n = lib.qmm_moe_workspace_bytes(tokens, gate.num_experts, top_k, gate.K, gate.N)
    if n < 0:
        _lib.check(int(n))
    return n


def moe_workspace(x: torch.Tensor, gate: ExpertWeights, top_k: int) -> torch.Tensor:
    """A workspace for moe calls of up to x.shape[0] tokens through experts like `gate`
    (reusable in stream order; its content does not matter)."""
    return torch.empty((_bytes(_lib.load(), x.shape[0], gate, top_k) + 3) // 4, dtype=torch.float32, device=x.device)


def moe(x: torch.Tensor, router_logits: torch.Tensor, gate: ExpertWeights, up: ExpertWeights, down: ExpertWeights,
        top_k: int, renormalize: bool = True, out=None, workspace=None) -> torch.Tensor:
    """The layer's output [tokens, hidden] for x [tokens, hidden] (at most 32 rows; any row
    stride that is a multiple of 8) and router_logits [tokens, experts] (qmm_moe): each token's
    top_k experts, softmax over them (renormalize) or over all, SwiGLU through gate, up and
    down."""
    lib = _lib.load()
    experts = gate.w_packed.size(0)
    if x.dim() != 2 or router_logits.shape != (x.size(0), experts):
        raise ValueError("moe: x %s must be [tokens, hidden], router_logits %s [tokens, %d]"
                         % (tuple(x.shape), tuple(router_logits.shape), experts))
    tokens, hidden = x.shape
    if hidden != gate.K:
        raise _lib.QmmError(-3, "moe: x has %d columns, the experts take %d" % (hidden, gate.K))
    code = _DTYPE_CODE.get(x.dtype, 0)
    if router_logits.dtype != x.dtype:
        raise _lib.QmmError(-2, "x and router_logits must share one dtype")
    xs, xl = x.stride()
    rs, rl = router_logits.stride()
    if tokens and ((xl != 1 and hidden > 1) or (rl != 1 and experts > 1)):
        raise _lib.QmmError(-4, "moe: the last stride of x and router_logits must be 1")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        assert out.dtype == x.dtype and out.shape == x.shape and (out.stride(1) == 1 or tokens == 0)
    if workspace is None:
        workspace = moe_workspace(x, gate, top_k)
    assert workspace.is_contiguous()
    same_device("moe", x, router_logits, out, workspace, gate.w_packed, gate.scales, gate.biases, up.w_packed, up.scales,
                up.biases, down.w_packed, down.scales, down.biases)
    g, u, d = _stack(gate), _stack(up), _stack(down)
    pointer = ctypes.pointer
    if tokens <= 1:                      # one row's strides may be anything
        xs, rs, ys = hidden, experts, hidden
    else:
        ys = out.stride(0)
    args = _lib.MoeDesc(x.data_ptr(), xs, router_logits.data_ptr(), rs, tokens, top_k, int(renormalize), code,
                        pointer(g), pointer(u), pointer(d), ys)
    _lib.check(lib.qmm_moe(ctypes.byref(args), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, raw_stream(x)))
    return out
