"""The mixture-of-experts layer for a few tokens (qmm_moe).  Argument marshalling only, like
api.py."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import ExpertWeights, _dtype_code, _stream


def _stack(w: ExpertWeights) -> _lib.ExpertStack:
    return _lib.ExpertStack(w.expert(0).desc(), w.num_experts, w.w_packed.stride(0), w.scales.stride(0))


def _bytes(tokens: int, gate: ExpertWeights, top_k: int) -> int:
    n = _lib.load().qmm_moe_workspace_bytes(tokens, gate.num_experts, top_k, gate.K, gate.N)
    if n < 0:
        _lib.check(int(n))
    return n


def moe_workspace(x: torch.Tensor, gate: ExpertWeights, top_k: int) -> torch.Tensor:
    """A workspace for moe calls of up to x.shape[0] tokens through experts like `gate`
    (reusable in stream order; its content does not matter)."""
    return torch.empty((_bytes(x.shape[0], gate, top_k) + 3) // 4, dtype=torch.float32, device=x.device)


def moe(x: torch.Tensor, router_logits: torch.Tensor, gate: ExpertWeights, up: ExpertWeights, down: ExpertWeights,
        top_k: int, renormalize: bool = True, out=None, workspace=None) -> torch.Tensor:
    """The layer's output [tokens, hidden] for x [tokens, hidden] (at most 32 rows; any row
    stride that is a multiple of 8) and router_logits [tokens, experts] (qmm_moe): each token's
    top_k experts, softmax over them (renormalize) or over all, SwiGLU through gate, up and
    down."""
    lib = _lib.load()
    if x.dim() != 2 or router_logits.dim() != 2 or router_logits.shape != (x.shape[0], gate.num_experts):
        raise ValueError("moe: x %s must be [tokens, hidden], router_logits %s [tokens, %d]"
                         % (tuple(x.shape), tuple(router_logits.shape), gate.num_experts))
    if x.shape[1] != gate.K:
        raise _lib.QmmError(-3, "moe: x has %d columns, the experts take %d" % (x.shape[1], gate.K))
    if router_logits.dtype != x.dtype:
        raise _lib.QmmError(-2, "x and router_logits must share one dtype")
    if x.numel() and (x.stride(1) != 1 or router_logits.stride(1) != 1):
        raise _lib.QmmError(-4, "moe: the last stride of x and router_logits must be 1")
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    assert y.dtype == x.dtype and y.shape == x.shape and (y.numel() == 0 or y.stride(1) == 1)
    stacks = [_stack(w) for w in (gate, up, down)]
    d = _lib.MoeDesc()
    d.x, d.x_stride = x.data_ptr(), x.stride(0) if x.shape[0] > 1 else x.shape[1]
    d.router_logits = router_logits.data_ptr()
    d.router_stride = router_logits.stride(0) if x.shape[0] > 1 else gate.num_experts
    d.tokens, d.top_k, d.renormalize, d.dtype = x.shape[0], top_k, int(renormalize), _dtype_code(x.dtype)
    d.gate, d.up, d.down = (ctypes.pointer(s) for s in stacks)
    d.y_stride = y.stride(0) if x.shape[0] > 1 else x.shape[1]
    ws = workspace
    if ws is None:
        ws = moe_workspace(x, gate, top_k)
    assert ws.is_contiguous()
    _lib.check(lib.qmm_moe(ctypes.byref(d), y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                           _stream(x.device)))
    return y
