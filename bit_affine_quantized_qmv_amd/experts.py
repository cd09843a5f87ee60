"""The mixture-of-experts layer for a few tokens (qmm_moe) and for any number (qmm_moe_prompt), and
products grouped by expert (qmm_grouped).  Argument marshalling only, like api.py."""
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
    return _layer("moe", moe_workspace, x, router_logits, gate, up, down, top_k, renormalize, out, workspace)


def _layer(who, make_workspace, x, router_logits, gate, up, down, top_k, renormalize, out, workspace):
    lib = _lib.load()
    experts = gate.w_packed.size(0)
    if x.dim() != 2 or router_logits.shape != (x.size(0), experts):
        raise ValueError("%s: x %s must be [tokens, hidden], router_logits %s [tokens, %d]"
                         % (who, tuple(x.shape), tuple(router_logits.shape), experts))
    tokens, hidden = x.shape
    if hidden != gate.K:
        raise _lib.QmmError(-3, "%s: x has %d columns, the experts take %d" % (who, hidden, gate.K))
    code = _DTYPE_CODE.get(x.dtype, 0)
    if router_logits.dtype != x.dtype:
        raise _lib.QmmError(-2, "x and router_logits must share one dtype")
    xs, xl = x.stride()
    rs, rl = router_logits.stride()
    if tokens and ((xl != 1 and hidden > 1) or (rl != 1 and experts > 1)):
        raise _lib.QmmError(-4, "%s: the last stride of x and router_logits must be 1" % who)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        assert out.dtype == x.dtype and out.shape == x.shape and (out.stride(1) == 1 or tokens == 0)
    if workspace is None:
        workspace = make_workspace(x, gate, top_k)
    assert workspace.is_contiguous()
    same_device(who, x, router_logits, out, workspace, gate.w_packed, gate.scales, gate.biases, up.w_packed, up.scales,
                up.biases, down.w_packed, down.scales, down.biases)
    g, u, d = _stack(gate), _stack(up), _stack(down)
    pointer = ctypes.pointer
    if tokens <= 1:                      # one row's strides may be anything
        xs, rs, ys = hidden, experts, hidden
    else:
        ys = out.stride(0)
    args = _lib.MoeDesc(x.data_ptr(), xs, router_logits.data_ptr(), rs, tokens, top_k, int(renormalize), code,
                        pointer(g), pointer(u), pointer(d), ys)
    call = lib.qmm_moe if who == "moe" else lib.qmm_moe_prompt
    _lib.check(call(ctypes.byref(args), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, raw_stream(x)))
    return out


def moe_prompt_workspace(x: torch.Tensor, gate: ExpertWeights, top_k: int) -> torch.Tensor:
    """A workspace for moe_prompt calls of up to x.shape[0] tokens through experts like `gate`
    (reusable in stream order; its content does not matter)."""
    n = _lib.load().qmm_moe_prompt_workspace_bytes(x.shape[0], gate.num_experts, top_k, gate.K, gate.N)
    if n < 0:
        _lib.check(int(n))
    return torch.empty((n + 3) // 4, dtype=torch.float32, device=x.device)


def moe_prompt(x: torch.Tensor, router_logits: torch.Tensor, gate: ExpertWeights, up: ExpertWeights,
               down: ExpertWeights, top_k: int, renormalize: bool = True, out=None, workspace=None) -> torch.Tensor:
    """The layer of moe for any number of tokens (qmm_moe_prompt): products grouped by expert on the
    matrix cores.  Arguments as moe's, the workspace moe_prompt_workspace's."""
    return _layer("moe_prompt", moe_prompt_workspace, x, router_logits, gate, up, down, top_k, renormalize, out,
                  workspace)


def grouped_workspace(x: torch.Tensor, experts: ExpertWeights) -> torch.Tensor:
    """A workspace for grouped_qmm calls of up to x.shape[0] rows (reusable in stream order; its
    content does not matter)."""
    w = _stack(experts)
    n = _lib.load().qmm_grouped_workspace_bytes(x.shape[0], ctypes.byref(w))
    if n < 0:
        _lib.check(int(n))
    return torch.empty((n + 3) // 4, dtype=torch.float32, device=x.device)


def grouped_qmm(x: torch.Tensor, experts: ExpertWeights, offsets: torch.Tensor, out=None,
                workspace=None) -> torch.Tensor:
    """y[r] = x[r] . W_e^T for the rows offsets[e] <= r < offsets[e + 1] of x [rows, K] (any row
    stride that is a multiple of 8; qmm_grouped); offsets int32 [experts + 1] on the GPU, ascending.
    Rows of no expert keep what `out` holds, zeros without one."""
    lib = _lib.load()
    if x.dim() != 2 or x.size(1) != experts.K:
        raise ValueError("grouped_qmm: x %s must be [rows, %d]" % (tuple(x.shape), experts.K))
    rows = x.size(0)
    if offsets.dtype != torch.int32 or not offsets.is_contiguous() or offsets.shape != (experts.num_experts + 1,):
        raise ValueError("grouped_qmm: offsets (%s %s) must be a contiguous int32 tensor of %d numbers"
                         % (offsets.dtype, tuple(offsets.shape), experts.num_experts + 1))
    if x.dtype != experts.scales.dtype:
        raise _lib.QmmError(-2, "x and the experts must share one dtype")
    xs, xl = x.stride()
    if rows and xl != 1 and experts.K > 1:
        raise _lib.QmmError(-4, "grouped_qmm: the last stride of x must be 1")
    if out is None:
        out = x.new_zeros((rows, experts.N))
    elif out.dtype != x.dtype or out.shape != (rows, experts.N) or (out.stride(1) != 1 and experts.N > 1 and rows):
        raise ValueError("grouped_qmm: out must be [%d, %d] of x's dtype, its last stride 1" % (rows, experts.N))
    if workspace is None:
        workspace = grouped_workspace(x, experts)
    if not workspace.is_contiguous():
        raise ValueError("grouped_qmm: the workspace must be contiguous")
    same_device("grouped_qmm", x, offsets, out, workspace, experts.w_packed, experts.scales, experts.biases)
    w = _stack(experts)
    if rows <= 1:                        # one row's strides may be anything
        xs, ys = experts.K, experts.N
    else:
        ys = out.stride(0)
    _lib.check(lib.qmm_grouped(x.data_ptr(), xs, rows, ctypes.byref(w), offsets.data_ptr(), out.data_ptr(), ys,
                               workspace.data_ptr(), workspace.nbytes, raw_stream(x)))
    return out
