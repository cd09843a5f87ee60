"""Sampling from logits (qmm_sample).  Argument marshalling only, like api.py."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _dtype_code, _stream

_WORKSPACE_BYTES = 190520    # per row


def sample_workspace(rows: int, device) -> torch.Tensor:
    """A workspace for sample calls of up to `rows` rows (reusable in stream order; its content
    does not matter)."""
    return torch.empty(_WORKSPACE_BYTES // 8 * max(rows, 1), dtype=torch.int64, device=device)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out_index=None,
           out_prob=None, workspace=None):
    """Draw one column per row of logits [rows, n] with the uniform numbers u [rows]
    (qmm_sample): (index int32 [rows], probability float32 [rows]).  temperature, top_k, top_p
    and min_p are numbers or device tensors [rows] (float32; top_k int32).  temperature 0 takes
    the largest logit; a row of nothing but NaN and -inf gives index -1 and probability 0."""
    lib = _lib.load()
    assert logits.dim() == 2 and (logits.numel() == 0 or logits.stride(1) == 1)
    rows, n = logits.shape
    assert u.dtype == torch.float32 and u.is_cuda and u.is_contiguous() and u.numel() == rows
    p = _lib.SampleParams()
    for name, value, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                               ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(value, torch.Tensor):
            assert value.dtype == dtype and value.is_cuda and value.is_contiguous() and value.numel() == rows, name
            setattr(p, name, value.data_ptr())
        else:
            setattr(p, name + "_all", value)
    idx = out_index if out_index is not None else torch.empty(rows, dtype=torch.int32, device=logits.device)
    prob = out_prob if out_prob is not None else torch.empty(rows, dtype=torch.float32, device=logits.device)
    assert idx.dtype == torch.int32 and idx.is_contiguous() and idx.numel() >= rows
    assert prob.dtype == torch.float32 and prob.is_contiguous() and prob.numel() >= rows
    ws = workspace if workspace is not None else sample_workspace(rows, logits.device)
    assert ws.is_contiguous() and ws.numel() * ws.element_size() >= _WORKSPACE_BYTES * rows
    _lib.check(lib.qmm_sample(logits.data_ptr(), _dtype_code(logits.dtype), rows, n,
                              logits.stride(0) if rows > 1 else n, ctypes.byref(p), u.data_ptr(), idx.data_ptr(),
                              prob.data_ptr(), ws.data_ptr(), _stream(logits.device)))
    return idx, prob
