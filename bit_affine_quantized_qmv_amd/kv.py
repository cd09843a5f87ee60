"""The 4-bit key/value cache and attention over it (qmm_kv_append, qmm_kv_read,
qmm_kv_attend).  Argument marshalling only, like api.py."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from .api import _DTYPE_CODE, _DTYPE_NAME, _stream


@dataclass
class KVCache:
    """`pages` pages of `page_size` token slots with one K and one V row of `head_dim` values
    per slot and kv head, 4-bit codes with a scale and bias in `dtype` per group.  `data` is
    int32 [pages, heads, words] in the library's own order."""
    data: torch.Tensor
    page_size: int
    head_dim: int
    group_size: int
    dtype: torch.dtype

    @property
    def pages(self) -> int:
        return self.data.shape[0]

    @property
    def heads(self) -> int:
        return self.data.shape[1]

    def desc(self) -> _lib.KVCacheDesc:
        assert self.data.dtype == torch.int32 and self.data.is_contiguous()
        assert self.data.shape[2] == _page_words(self.page_size, self.head_dim, self.group_size)
        return _lib.KVCacheDesc(self.data.data_ptr(), self.pages, self.page_size, self.heads, self.head_dim,
                                self.group_size, _DTYPE_CODE[self.dtype])


def _page_words(page_size: int, head_dim: int, group_size: int) -> int:
    return 2 * page_size * (head_dim // 8 + head_dim // group_size)


def kv_cache(pages: int, page_size: int, heads: int, head_dim: int, group_size: int = 64, dtype="bf16",
             device="cuda") -> KVCache:
    """An empty cache (zero-filled)."""
    if isinstance(dtype, str):
        dtype = _DTYPE_NAME[dtype]
    words = _page_words(page_size, head_dim, group_size)
    return KVCache(torch.zeros(pages, heads, words, dtype=torch.int32, device=device), page_size, head_dim,
                   group_size, dtype)


def _check_slots(slots: torch.Tensor) -> None:
    assert slots.dtype == torch.int32 and slots.is_cuda and slots.is_contiguous() and slots.dim() == 1


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k[t, h] and v[t, h] ([tokens, heads, head_dim], any token and head strides)
    into slot slots[t] of every head; slots outside the cache are skipped."""
    lib = _lib.load()
    _check_slots(slots)
    want = (slots.numel(), cache.heads, cache.head_dim)
    if tuple(k.shape) != want or tuple(v.shape) != want:
        raise ValueError("kv_append: k %s and v %s must be [tokens, heads, head_dim] = %s"
                         % (tuple(k.shape), tuple(v.shape), want))
    if k.dtype != cache.dtype or v.dtype != cache.dtype:
        raise _lib.QmmError(-2, "k, v and the cache must share one dtype")
    if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
        raise _lib.QmmError(-4, "kv_append: the last stride of k and v must be 1")
    _lib.check(lib.qmm_kv_append(ctypes.byref(cache.desc()), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                 v.stride(0), v.stride(1), slots.data_ptr(), slots.numel(), _stream(k.device)))


def kv_read(cache: KVCache, slots: torch.Tensor, out_k=None, out_v=None):
    """The K and V rows that the cache stands for at `slots`: two [count, heads, head_dim]
    tensors (NaN rows for slots outside the cache)."""
    lib = _lib.load()
    _check_slots(slots)
    shape = (slots.numel(), cache.heads, cache.head_dim)
    k = out_k if out_k is not None else torch.empty(shape, dtype=cache.dtype, device=slots.device)
    v = out_v if out_v is not None else torch.empty(shape, dtype=cache.dtype, device=slots.device)
    for t in (k, v):
        assert t.dtype == cache.dtype and t.is_contiguous() and tuple(t.shape) == shape
    _lib.check(lib.qmm_kv_read(ctypes.byref(cache.desc()), slots.data_ptr(), slots.numel(), k.data_ptr(),
                               v.data_ptr(), _stream(slots.device)))
    return k, v


def _attend_desc(q: torch.Tensor, cache: KVCache, max_length: int) -> _lib.KVAttendDesc:
    if q.dim() != 4 or q.shape[3] != cache.head_dim:
        raise ValueError("kv_attend: q %s must be [batch, q_len, q_heads, %d]" % (tuple(q.shape), cache.head_dim))
    d = _lib.KVAttendDesc()
    d.q = q.data_ptr()
    d.q_batch_stride, d.q_token_stride, d.q_head_stride = q.stride(0), q.stride(1), q.stride(2)
    d.batch, d.q_len, d.q_heads = q.shape[0], q.shape[1], q.shape[2]
    d.causal = 1
    d.max_length = max_length
    d.max_blocks = d.table_stride = -(-max_length // cache.page_size)
    return d


def kv_attend_workspace(q: torch.Tensor, cache: KVCache, max_length: int) -> torch.Tensor:
    """A workspace for kv_attend calls with queries shaped like q over sequences of up to
    max_length tokens (reusable in stream order; its content does not matter)."""
    n = _lib.load().qmm_kv_attend_workspace_bytes(ctypes.byref(cache.desc()),
                                                  ctypes.byref(_attend_desc(q, cache, max_length)))
    if n < 0:
        _lib.check(int(n))
    return torch.empty(max(n, 16) // 4, dtype=torch.float32, device=q.device)


def kv_attend(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor, scale=None,
              causal: bool = True, window: int = 0, max_length=None, out=None, workspace=None) -> torch.Tensor:
    """Attention of q [batch, q_len, q_heads, head_dim] (any strides, the last 1) over the
    cached tokens of each sequence (qmm_kv_attend): the queries are the sequence's last q_len
    tokens; block_table int32 [batch, blocks] names its pages, lengths int32 [batch] its token
    counts.  scale defaults to head_dim ** -0.5; max_length (an upper bound on the lengths,
    known on the host) defaults to what the block table can hold; a smaller one launches less.
    Queries that see no token give zeros."""
    lib = _lib.load()
    assert block_table.dtype == torch.int32 and block_table.dim() == 2
    assert block_table.is_cuda and (block_table.numel() == 0 or block_table.stride(1) == 1)
    assert lengths.dtype == torch.int32 and lengths.is_cuda and lengths.is_contiguous()
    if block_table.shape[0] != q.shape[0] or lengths.numel() != q.shape[0]:
        raise ValueError("kv_attend: %d sequences, %d block table rows, %d lengths"
                         % (q.shape[0], block_table.shape[0], lengths.numel()))
    if q.dtype != cache.dtype:
        raise _lib.QmmError(-2, "q and the cache must share one dtype")
    if q.numel() and q.stride(3) != 1:
        raise _lib.QmmError(-4, "kv_attend: the last stride of q must be 1")
    blocks = block_table.shape[1]
    d = _attend_desc(q, cache, blocks * cache.page_size if max_length is None else max_length)
    d.scale = cache.head_dim ** -0.5 if scale is None else scale
    d.causal, d.window = int(causal), window
    d.block_table, d.max_blocks = block_table.data_ptr(), blocks
    d.table_stride = block_table.stride(0) if block_table.shape[0] > 1 else blocks
    d.lengths = lengths.data_ptr()
    y = out if out is not None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    assert y.dtype == q.dtype and y.is_contiguous() and y.shape == q.shape
    cd = cache.desc()
    if workspace is None:
        n = lib.qmm_kv_attend_workspace_bytes(ctypes.byref(cd), ctypes.byref(d))
        if n < 0:
            _lib.check(int(n))
        workspace = torch.empty(n // 4, dtype=torch.float32, device=q.device) if n else None
    ws, size = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    _lib.check(lib.qmm_kv_attend(ctypes.byref(cd), ctypes.byref(d), y.data_ptr(), ws, size, _stream(q.device)))
    return y
