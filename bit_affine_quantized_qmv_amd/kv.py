"""The 4-bit key/value cache and attention over it (qmm_kv_append, qmm_kv_read,
qmm_kv_attend).  Argument marshalling only, like api.py; these calls are made once per layer
and token, so each tensor's shape and strides are read once."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib, api
from .api import _DTYPE_CODE, _DTYPE_NAME

_byref = ctypes.byref


def raw_stream(t: torch.Tensor) -> int:
    """The current stream of t's device, which has to be the current one, as an address."""
    index = t.get_device()
    if api._gpus != 1:
        api.check_current(index)
    return torch._C._cuda_getCurrentRawStream(index)


def same_device(who: str, first: torch.Tensor, *others) -> None:
    """The tensors of one call are on one GPU (None: not given)."""
    device = first.get_device()
    for t in (first,) + others:
        if t is not None and (device < 0 or t.get_device() != device):
            raise ValueError("%s: a tensor is on %s, another on %s; all must be on one GPU"
                             % (who, first.device, t.device))


@dataclass(frozen=True)
class KVCache:
    """`pages` pages of `page_size` token slots with one K and one V row of `head_dim` values
    per slot and kv head, 4-bit codes with a scale and bias in `dtype` per group.  `data` is
    int32 [pages, heads, words] in the library's own order; it stays where it is for the
    cache's life."""
    data: torch.Tensor
    page_size: int
    head_dim: int
    group_size: int
    dtype: torch.dtype

    def __post_init__(self):
        pages, heads, words = self.data.shape
        assert self.data.dtype == torch.int32 and self.data.is_contiguous()
        assert words == _page_words(self.page_size, self.head_dim, self.group_size)
        object.__setattr__(self, "pages", pages)
        object.__setattr__(self, "heads", heads)
        object.__setattr__(self, "_desc", _lib.KVCacheDesc(self.data.data_ptr(), pages, self.page_size, heads,
                                                           self.head_dim, self.group_size, _DTYPE_CODE[self.dtype]))

    def desc(self) -> _lib.KVCacheDesc:
        return self._desc


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


def _check_slots(slots: torch.Tensor) -> int:
    assert slots.dtype == torch.int32 and slots.is_cuda and slots.dim() == 1 and slots.is_contiguous()
    return slots.numel()


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k[t, h] and v[t, h] ([tokens, heads, head_dim], any token and head strides)
    into slot slots[t] of every head; slots outside the cache are skipped."""
    lib = _lib.load()
    tokens = _check_slots(slots)
    same_device("kv_append", slots, k, v, cache.data)
    want = (tokens, cache.heads, cache.head_dim)
    if k.shape != want or v.shape != want:
        raise ValueError("kv_append: k %s and v %s must be [tokens, heads, head_dim] = %s"
                         % (tuple(k.shape), tuple(v.shape), want))
    if k.dtype != cache.dtype or v.dtype != cache.dtype:
        raise _lib.QmmError(-2, "k, v and the cache must share one dtype")
    kt, kh, kd = k.stride()
    vt, vh, vd = v.stride()
    if tokens and (kd != 1 or vd != 1):
        raise _lib.QmmError(-4, "kv_append: the last stride of k and v must be 1")
    _lib.check(lib.qmm_kv_append(_byref(cache._desc), k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(),
                                 tokens, raw_stream(slots)))


def kv_read(cache: KVCache, slots: torch.Tensor, out_k=None, out_v=None):
    """The K and V rows that the cache stands for at `slots`: two [count, heads, head_dim]
    tensors (NaN rows for slots outside the cache)."""
    lib = _lib.load()
    count = _check_slots(slots)
    shape = (count, cache.heads, cache.head_dim)
    out = []
    for t in (out_k, out_v):
        if t is None:
            t = slots.new_empty(shape, dtype=cache.dtype)
        else:
            assert t.dtype == cache.dtype and t.is_contiguous() and t.shape == shape
        out.append(t)
    same_device("kv_read", slots, out[0], out[1], cache.data)
    _lib.check(lib.qmm_kv_read(_byref(cache._desc), slots.data_ptr(), count, out[0].data_ptr(), out[1].data_ptr(),
                               raw_stream(slots)))
    return out[0], out[1]


def _attend_desc(q, cache, scale, causal, window, table, table_stride, blocks, lengths, max_length):
    if q.dim() != 4 or q.size(3) != cache.head_dim:
        raise ValueError("kv_attend: q %s must be [batch, q_len, q_heads, %d]" % (tuple(q.shape), cache.head_dim))
    batch, q_len, heads, _ = q.shape
    sb, st, sh, sd = q.stride()
    if sd != 1 and q.numel():
        raise _lib.QmmError(-4, "kv_attend: the last stride of q must be 1")
    return _lib.KVAttendDesc(q.data_ptr(), sb, st, sh, batch, q_len, heads, causal, window, scale, table, table_stride,
                             blocks, lengths, max_length)


def _workspace_bytes(lib, cache, d) -> int:
    n = lib.qmm_kv_attend_workspace_bytes(_byref(cache._desc), _byref(d))
    if n < 0:
        _lib.check(int(n))
    return n


def kv_attend_workspace(q: torch.Tensor, cache: KVCache, max_length: int) -> torch.Tensor:
    """A workspace for kv_attend calls with queries shaped like q over sequences of up to
    max_length tokens (reusable in stream order; its content does not matter)."""
    blocks = -(-max_length // cache.page_size)
    n = _workspace_bytes(_lib.load(), cache, _attend_desc(q, cache, 1.0, 1, 0, None, blocks, blocks, None, max_length))
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
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_cuda
    assert lengths.dtype == torch.int32 and lengths.is_cuda and lengths.is_contiguous()
    rows, blocks = block_table.shape
    row_stride, last = block_table.stride()
    assert last == 1 or blocks <= 1
    batch = q.size(0)
    if rows != batch or lengths.numel() != batch:
        raise ValueError("kv_attend: %d sequences, %d block table rows, %d lengths" % (batch, rows, lengths.numel()))
    if q.dtype != cache.dtype:
        raise _lib.QmmError(-2, "q and the cache must share one dtype")
    d = _attend_desc(q, cache, cache.head_dim ** -0.5 if scale is None else scale, int(causal), window,
                     block_table.data_ptr(), row_stride if rows > 1 else blocks, blocks, lengths.data_ptr(),
                     blocks * cache.page_size if max_length is None else max_length)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        assert out.dtype == q.dtype and out.is_contiguous() and out.shape == q.shape
    if workspace is None:
        n = _workspace_bytes(lib, cache, d)
        workspace = q.new_empty(n // 4, dtype=torch.float32) if n else None
    same_device("kv_attend", q, cache.data, block_table, lengths, out, workspace)
    ws, size = (workspace.data_ptr(), workspace.nbytes) if workspace is not None else (None, 0)
    _lib.check(lib.qmm_kv_attend(_byref(cache._desc), _byref(d), out.data_ptr(), ws, size, raw_stream(q)))
    return out
