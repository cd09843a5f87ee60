"""Sampling from logits (qmm_sample).  Argument marshalling only, like api.py."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _dtype_code
from .kv import raw_stream, same_device

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
    rows, n = logits.shape
    stride, last = logits.stride()
    assert last == 1 or rows == 0 or n == 1
    assert u.dtype == torch.float32 and u.is_cuda and u.is_contiguous() and u.numel() == rows
    arrays, numbers = [], []
    for name, value, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                               ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(value, torch.Tensor):
            assert value.dtype == dtype and value.is_cuda and value.is_contiguous() and value.numel() == rows, name
            arrays.append(value.data_ptr())
            numbers.append(0)
        else:
            arrays.append(None)
            numbers.append(value)
    p = _lib.SampleParams(*arrays, *numbers)
    if out_index is None:
        out_index = u.new_empty(rows, dtype=torch.int32)
    else:
        assert out_index.dtype == torch.int32 and out_index.is_contiguous() and out_index.numel() >= rows
    if out_prob is None:
        out_prob = u.new_empty(rows)
    else:
        assert out_prob.dtype == torch.float32 and out_prob.is_contiguous() and out_prob.numel() >= rows
    if workspace is None:
        workspace = sample_workspace(rows, logits.device)
    assert workspace.is_contiguous() and workspace.nbytes >= _WORKSPACE_BYTES * rows
    same_device("sample", u, logits, out_index, out_prob, workspace)
    _lib.check(lib.qmm_sample(logits.data_ptr(), _dtype_code(logits.dtype), rows, n, stride if rows > 1 else n,
                              ctypes.byref(p), u.data_ptr(), out_index.data_ptr(), out_prob.data_ptr(),
                              workspace.data_ptr(), raw_stream(u)))
    return out_index, out_prob
