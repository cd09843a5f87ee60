"""Trees of drafted tokens over the 4-bit key/value cache, and the cache's pages (qmm_tree_mask,
qmm_kv_attend_tree, qmm_tree_accept, qmm_kv_move, qmm_kv_fork, qmm_kv_copy_pages).  Argument
marshalling only, like api.py."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .kv import KVCache, _attend_desc, raw_stream, same_device

_byref = ctypes.byref
_int32 = torch.int32


def _ints(who: str, name: str, t: torch.Tensor, *shape) -> int:
    """The row stride of an int32 GPU tensor of this shape (None: any), its last stride 1; that of a
    single row may be anything."""
    sizes = t.shape
    fits = t.dtype == _int32 and t.is_cuda and len(sizes) == len(shape)
    if fits and sizes != shape:
        for n, m in zip(shape, sizes):
            fits = fits and (n is None or n == m)
    if not fits:
        raise ValueError("%s: %s (%s %s on %s) must be an int32 GPU tensor of shape %s"
                         % (who, name, t.dtype, tuple(sizes), t.device, ["any" if n is None else n for n in shape]))
    strides = t.stride()
    if strides[-1] != 1 and sizes[-1] > 1:
        raise _lib.QmmError(-4, "%s: the last stride of %s must be 1" % (who, name))
    return strides[0] if sizes[0] > 1 else sizes[-1]


def tree_mask(parents: torch.Tensor, window: int = 0):
    """Which nodes each node of the trees parents int32 [batch, nodes] sees (qmm_tree_mask):
    (mask int32 [batch, nodes, ceil(nodes / 32)], depth int32 [batch, nodes]).  parents[i] is an
    earlier node, -1 for a root, less for what is no node; window limits how many nodes of its own
    path a node sees.  Node i of a sequence whose tree starts at position c stands for position
    c + depth[i]."""
    lib = _lib.load()
    stride = _ints("tree_mask", "parents", parents, None, None)
    batch, nodes = parents.shape
    mask = parents.new_empty((batch, nodes, (nodes + 31) // 32))
    depth = parents.new_empty((batch, nodes))
    _lib.check(lib.qmm_tree_mask(parents.data_ptr(), stride, batch, nodes, window, mask.data_ptr(),
                                 depth.data_ptr(), raw_stream(parents)))
    return mask, depth


def _tree_workspace_bytes(lib, cache, d) -> int:
    n = lib.qmm_kv_attend_tree_workspace_bytes(_byref(cache._desc), _byref(d))
    if n < 0:
        _lib.check(int(n))
    return n


def kv_attend_tree_workspace(q: torch.Tensor, cache: KVCache, max_length: int) -> torch.Tensor:
    """A workspace for kv_attend_tree calls with queries shaped like q over sequences of up to
    max_length tokens (reusable in stream order; its content does not matter)."""
    blocks = -(-max_length // cache.page_size)
    n = _tree_workspace_bytes(_lib.load(), cache,
                              _attend_desc(q, cache, 1.0, 1, 0, None, blocks, blocks, None, max_length))
    return torch.empty(max(n, 16) // 4, dtype=torch.float32, device=q.device)


def kv_attend_tree(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor, mask: torch.Tensor,
                   depth=None, scale=None, window: int = 0, max_length=None, out=None, workspace=None) -> torch.Tensor:
    """Attention of drafted trees (qmm_kv_attend_tree): q [batch, nodes, q_heads, head_dim] (any
    strides, the last 1) are the trees' nodes, the last `nodes` tokens of each sequence.  A node
    sees the tokens before its tree (with a window those near enough to its depth) and the nodes of
    its row of mask; mask and depth are tree_mask's, with the same window, or the caller's own (any
    depths from 0 on).  What is no node gives zeros.  The other arguments are kv_attend's."""
    lib = _lib.load()
    if q.dim() != 4:
        raise ValueError("kv_attend_tree: q %s must be [batch, nodes, q_heads, head_dim]" % (tuple(q.shape),))
    batch, nodes = q.shape[:2]
    table_stride = _ints("kv_attend_tree", "block_table", block_table, batch, None)
    _ints("kv_attend_tree", "lengths", lengths, batch)
    _ints("kv_attend_tree", "mask", mask, batch, nodes, (nodes + 31) // 32)
    if depth is not None:
        _ints("kv_attend_tree", "depth", depth, batch, nodes)
    if not mask.is_contiguous() or (depth is not None and not depth.is_contiguous()):
        raise _lib.QmmError(-4, "kv_attend_tree: mask and depth must be contiguous")
    if q.dtype != cache.dtype:
        raise _lib.QmmError(-2, "q and the cache must share one dtype")
    blocks = block_table.size(1)
    d = _attend_desc(q, cache, cache.head_dim ** -0.5 if scale is None else scale, 1, window, block_table.data_ptr(),
                     table_stride, blocks, lengths.data_ptr(),
                     blocks * cache.page_size if max_length is None else max_length)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.dtype != q.dtype or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("kv_attend_tree: out must be contiguous, of q's shape and dtype")
    if workspace is None:
        n = _tree_workspace_bytes(lib, cache, d)
        workspace = q.new_empty(n // 4, dtype=torch.float32) if n else None
    same_device("kv_attend_tree", q, cache.data, block_table, lengths, mask, depth, out, workspace)
    ws, size = (workspace.data_ptr(), workspace.nbytes) if workspace is not None else (None, 0)
    _lib.check(lib.qmm_kv_attend_tree(_byref(cache._desc), _byref(d), mask.data_ptr(),
                                      depth.data_ptr() if depth is not None else None, out.data_ptr(), ws, size,
                                      raw_stream(q)))
    return out


def tree_accept(parents: torch.Tensor, tokens: torch.Tensor, sampled: torch.Tensor):
    """The path of each tree that verification accepts (qmm_tree_accept), from its parents, drafted
    and sampled tokens, int32 [batch, nodes] each: (path int32 [batch, nodes], -1 after its end,
    count int32 [batch], last int32 [batch]: the token sampled after the path's end)."""
    lib = _lib.load()
    parents_stride = _ints("tree_accept", "parents", parents, None, None)
    shape = batch, nodes = parents.shape
    tokens_stride = _ints("tree_accept", "tokens", tokens, batch, nodes)
    sampled_stride = _ints("tree_accept", "sampled", sampled, batch, nodes)
    same_device("tree_accept", parents, tokens, sampled)
    path, count, last = parents.new_empty(shape), parents.new_empty(batch), parents.new_empty(batch)
    a = _lib.TreeAcceptDesc(parents.data_ptr(), tokens.data_ptr(), sampled.data_ptr(), parents_stride, tokens_stride,
                            sampled_stride, batch, nodes)
    _lib.check(lib.qmm_tree_accept(_byref(a), path.data_ptr(), count.data_ptr(), last.data_ptr(), raw_stream(parents)))
    return path, count, last


def kv_move(cache: KVCache, block_table: torch.Tensor, index: torch.Tensor, start: torch.Tensor, origin=None,
            to_table=None) -> None:
    """Move the cached rows at positions origin[n] + index[n, i] (origin None: 0) of sequence n to
    positions start[n] + i (qmm_kv_move); negative indices move nothing.  Within the sequence's own
    pages the indices have to ascend and no row may move up; with to_table the rows go to its pages,
    of which the call may read none."""
    lib = _lib.load()
    index_stride = _ints("kv_move", "index", index, None, None)
    batch, count = index.shape
    table_stride = _ints("kv_move", "block_table", block_table, batch, None)
    _ints("kv_move", "start", start, batch)
    if origin is not None:
        _ints("kv_move", "origin", origin, batch)
    to, to_stride, to_blocks = None, 0, 0
    if to_table is not None:
        to_stride = _ints("kv_move", "to_table", to_table, batch, None)
        to, to_blocks = to_table.data_ptr(), to_table.size(1)
    same_device("kv_move", index, block_table, start, origin, to_table, cache.data)
    a = _lib.KVMoveDesc(block_table.data_ptr(), table_stride, block_table.size(1), to, to_stride, to_blocks,
                        index.data_ptr(), index_stride, batch, count,
                        origin.data_ptr() if origin is not None else None, start.data_ptr())
    _lib.check(lib.qmm_kv_move(_byref(cache._desc), _byref(a), raw_stream(index)))


def kv_copy_pages(cache: KVCache, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Copy pages src[i] to dst[i] (int32; qmm_kv_copy_pages); pairs with a page outside the cache
    are skipped.  The dst are distinct and no src."""
    lib = _lib.load()
    _ints("kv_copy_pages", "src", src, None)
    _ints("kv_copy_pages", "dst", dst, src.size(0))
    same_device("kv_copy_pages", src, dst, cache.data)
    _lib.check(lib.qmm_kv_copy_pages(_byref(cache._desc), src.data_ptr(), dst.data_ptr(), src.size(0), raw_stream(src)))


def kv_fork(refs: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor, parents: torch.Tensor, page_size: int,
            want=None, blocks=None):
    """Block tables that continue others, begin, grow, are cut back or end (qmm_kv_fork).  refs
    int32 [pages] counts the table entries that name each page and is brought up to date.  Row i of
    the new table [rows, blocks] (blocks: as many as the old one has) continues row parents[i] of
    block_table (outside it: begins empty) with room for want[i] tokens (None: its length); the pages
    from its first min(length, want[i]) tokens on are its own to write to.  Returns
    (table, copy_src, copy_dst, short): the pages to copy with kv_copy_pages in every layer's cache
    (-1: none), and int32 [1], how many entries got no page or no place in the table."""
    lib = _lib.load()
    _ints("kv_fork", "refs", refs, None)
    table_stride = _ints("kv_fork", "block_table", block_table, None, None)
    batch, old_blocks = block_table.shape
    _ints("kv_fork", "lengths", lengths, batch)
    _ints("kv_fork", "parents", parents, None)
    rows = parents.size(0)
    if want is not None:
        _ints("kv_fork", "want", want, rows)
    if blocks is None:
        blocks = old_blocks
    table = parents.new_empty((rows, max(blocks, 0)))
    pairs = parents.new_empty(2 * rows + 1)
    at = pairs.data_ptr()
    a = _lib.KVForkDesc(refs.data_ptr(), refs.size(0), page_size, block_table.data_ptr(), table_stride,
                        old_blocks, lengths.data_ptr(), batch, parents.data_ptr(),
                        want.data_ptr() if want is not None else None, rows, table.data_ptr(), blocks, blocks)
    n = lib.qmm_kv_fork_workspace_bytes(_byref(a))
    if n < 0:
        _lib.check(int(n))
    workspace = parents.new_empty(n // 4)
    same_device("kv_fork", refs, block_table, lengths, parents, want)
    _lib.check(lib.qmm_kv_fork(_byref(a), at, at + 4 * rows, at + 8 * rows, workspace.data_ptr(), n, raw_stream(refs)))
    return table, pairs[:rows], pairs[rows:2 * rows], pairs[2 * rows:]
