"""Trees, moves, page copies, forks and grouped products at their largest sizes, and page work in a
replayed graph and on another stream."""
import numpy as np
import pytest
import torch

import synth
from fork_testlib import cut_inputs, fork_rule
from qmm_testlib import half_bits, require_gpu, values
from test_gpu_grouped import check, offsets_of, product, reference, rounded
from test_gpu_kv_cache import _rows
from test_gpu_moe import stack
from test_gpu_tree import _ints

pytestmark = pytest.mark.gpu


def test_a_pool_past_32_bit_offsets():
    """The same work in the first pages of a small pool and in the last ones of a pool of more than 2^31
    words: the same bits."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    page, heads, dim, group, n, last = 64, 8, 128, 32, 300, 110000
    if torch.cuda.mem_get_info(dev)[0] < 16 << 30:
        pytest.skip("needs 16 GB of free GPU memory")
    small = q.kv_cache(30, page, heads, dim, group, "bf16", dev)
    large = q.kv_cache(last, page, heads, dim, group, "bf16", dev)
    assert large.data.numel() > 2 ** 31
    blocks = -(-n // page)
    k, v = (_rows((n, heads, dim), "bf16", seed).to(dev) for seed in (31, 32))
    results = []
    for cache, at in ((small, torch.arange(30)), (large, last - 1 - torch.arange(30))):
        at = at.to(torch.int32).to(dev)
        table, to = at[None, :blocks].contiguous(), at[None, blocks:2 * blocks].contiguous()
        j = torch.arange(n, device=dev)
        slots, moved = ((t[0, j // page] * page + j % page).int() for t in (table, to))
        q.kv_append(cache, k, v, slots)
        out = []
        for nodes in (20, 80):                                       # 40 rows per cached head, and 320
            parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device=dev)[None]
            mask, depth = q.tree_mask(parents)
            for heads_q in (2 * heads, 4 * heads):
                out.append(q.kv_attend_tree(_rows((1, nodes, heads_q, dim), "bf16", 33).to(dev), cache, table,
                                            _ints([n], dev), mask, depth))
        index = _ints([[3, 250, 7, 7, 299, 0]], dev)
        q.kv_append(cache, v, k, moved)
        q.kv_move(cache, table, index, _ints([130], dev), to_table=to)
        q.kv_move(cache, to, _ints([[1, 2, 90, 150]], dev), _ints([20], dev), origin=_ints([20], dev))
        q.kv_copy_pages(cache, at[blocks:blocks + 2].contiguous(), at[20:22].contiguous())
        copied = (at[20:22, None] * page + torch.arange(page, dtype=torch.int32, device=dev)).flatten()
        results.append(out + [*q.kv_read(cache, slots), *q.kv_read(cache, moved), *q.kv_read(cache, copied)])
    for a, b in zip(*results):
        assert not torch.isnan(a.float()).any() and torch.equal(a, b)


def test_the_largest_batch():
    """65535 trees of two nodes: masks, attention, acceptance and moves, against those of a few."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    batch, nodes, dim, page = 65535, 2, 64, 16
    cache = q.kv_cache(batch, page, 1, dim, 32, "bf16", dev)
    table = torch.arange(batch, dtype=torch.int32, device=dev).flip(0)[:, None].contiguous()
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(2, page + 1, (batch,), generator=g).to(torch.int32).to(dev)
    k, v = (torch.randn(batch * page, 1, dim, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    q.kv_append(cache, k, v, torch.arange(batch * page, dtype=torch.int32, device=dev))
    parents = torch.tensor([-1, 0], dtype=torch.int32, device=dev).expand(batch, 2).contiguous()
    parents[::7, 1] = -2
    queries = torch.randn(batch, nodes, 2, dim, generator=g).to(torch.bfloat16).to(dev)
    mask, depth = q.tree_mask(parents)
    y = q.kv_attend_tree(queries, cache, table, lengths, mask, depth)
    tokens, sampled = (torch.randint(0, 2, (batch, nodes), generator=g).to(torch.int32).to(dev) for _ in range(2))
    path, count, last = q.tree_accept(parents, tokens, sampled)
    follows = (parents[:, 1] == 0) & (tokens[:, 1] == sampled[:, 0])
    assert torch.equal(count, 1 + follows.int()) and torch.equal(path[:, 0], torch.zeros_like(count))
    assert torch.equal(path[:, 1], follows.int() * 2 - 1)
    assert torch.equal(last, torch.where(follows, sampled[:, 1], sampled[:, 0]))
    some = torch.cat([torch.arange(40), torch.arange(batch - 40, batch)]).to(dev)
    few = q.kv_attend_tree(queries[some], cache, table[some].contiguous(), lengths[some], mask[some].contiguous())
    assert torch.equal(few, y[some]) and torch.isfinite(y.float()).all()
    before = [t.clone() for t in q.kv_read(cache, torch.arange(batch * page, dtype=torch.int32, device=dev))]
    q.kv_move(cache, table, _ints([[1]], dev).expand(batch, 1).contiguous(), torch.zeros_like(lengths))
    after = q.kv_read(cache, torch.arange(batch * page, dtype=torch.int32, device=dev))
    for a, b in zip(before, after):
        a = a.view(batch, page, dim)
        a[:, 0] = a[:, 1]
        assert torch.equal(a.view_as(b), b)


def test_moves_and_copies_of_more_than_a_grid():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    page, blocks, dim = 65536, 66, 64
    cache = q.kv_cache(blocks + 1, page, 1, dim, 64, "fp16", dev)
    count = 64 * 65535 + 70000                           # steps of 64 positions that workgroups take twice
    where = [0, 5, 64 * 65535 - 1, 64 * 65535, 64 * 65535 + 3, count - 1]
    source = [3, 77, 12345, 9, 40000, 65535]
    rows = _rows((len(source), 1, dim), "fp16", 3).to(dev)
    q.kv_append(cache, rows, rows.flip(0), _ints([blocks * page + s for s in source], dev))
    index = torch.full((1, count), -1, dtype=torch.int32, device=dev)
    index[0, where] = _ints(source, dev)
    table, to = _ints([[blocks]], dev), torch.arange(blocks, dtype=torch.int32, device=dev).flip(0)[None].contiguous()
    q.kv_move(cache, table, index, _ints([2], dev), to_table=to)
    slots = [(blocks - 1 - (w + 2) // page) * page + (w + 2) % page for w in where]
    kept = [i for i, w in enumerate(where) if w + 2 < blocks * page]
    got_k, got_v = q.kv_read(cache, _ints([slots[i] for i in kept], dev))
    want_k, want_v = q.kv_read(cache, _ints([blocks * page + source[i] for i in kept], dev))
    assert len(kept) == 6 and torch.equal(got_k, want_k) and torch.equal(got_v, want_v)
    assert np.count_nonzero(half_bits(got_k).any(-1)) == 6
    assert int((cache.data[:blocks] != 0).any(2).sum()) == len({s // page for s in slots})
    # more pairs than a grid has rows; all but a few are none
    pool = q.kv_cache(50, 16, 2, dim, 64, "fp16", dev)
    pool.data.copy_(torch.arange(pool.data.numel(), dtype=torch.int32).view_as(pool.data))
    src, dst = (torch.full((70000,), -1, dtype=torch.int32, device=dev) for _ in range(2))
    at = torch.tensor([0, 65534, 65535, 65536, 69999], device=dev)
    src[at], dst[at] = _ints([1, 3, 5, 7, 9], dev), _ints([20, 30, 40, 48, 49], dev)
    want = pool.data.clone()
    want[[20, 30, 40, 48, 49]] = want[[1, 3, 5, 7, 9]]
    q.kv_copy_pages(pool, src, dst)
    assert torch.equal(pool.data, want)


def test_forks_of_the_most_rows():
    """65535 rows of 65535 sequences, one block each, then all of them from the first ten."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    n, pages = 65535, 140000
    g = np.random.RandomState(1)
    table = g.permutation(pages)[:n].astype(np.int32)
    lengths = g.randint(0, 17, n).astype(np.int32)
    refs = np.zeros(pages, np.int32)
    refs[table] = 1
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
    d_refs = t(refs)
    new, src, dst, short = q.kv_fork(d_refs, t(table)[:, None], t(lengths), torch.arange(n, dtype=torch.int32, device=dev).flip(0),
                                     16, t(np.full(n, 16, np.int32)))
    assert torch.equal(new[:, 0].flip(0), t(table)) and short.item() == 0 and torch.equal(d_refs, t(refs))
    assert (src == -1).all() and (dst == -1).all()
    parents = g.randint(0, 10, n)
    keep = g.randint(0, 17, n)
    new, src, dst, short = q.kv_fork(d_refs, new, t(lengths[::-1].copy()), t(parents.astype(np.int32)), 16, t(keep.astype(np.int32)))
    got = new[:, 0].cpu().numpy()
    kept = np.minimum(keep, lengths[::-1][parents])
    whole = kept == 16
    assert (got[whole] == table[::-1][parents[whole]]).all() and (got[keep == 0] == -1).all() and short.item() == 0
    counts = np.bincount(got[got >= 0], minlength=pages)
    assert np.array_equal(counts, d_refs.cpu().numpy()) and (counts[got[~whole & (keep > 0)]] == 1).all()
    copies = dst.cpu().numpy() >= 0
    assert (src.cpu().numpy()[copies] == table[::-1][parents[copies]]).all() and np.array_equal(dst.cpu().numpy()[copies], got[copies])
    first = np.array([np.flatnonzero(parents == p)[0] for p in range(10)])
    part = (kept > 0) & (kept < 16)
    assert not copies[~part].any() and copies[np.setdiff1d(np.flatnonzero(part), first)].all()


def test_the_most_rows_of_a_product():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    rows, dtype = 2 ** 20, "bf16"
    w = stack(8, 32, 32, 4, dtype, 3, 5, dev)
    x = synth.normal_x((rows, 32), dtype, seed=1)
    counts = [700001, 0, rows - 700001 - 3]                          # the last three rows are nobody's
    offsets = offsets_of(counts)
    y = q.grouped_qmm(x.to(dev), w, offsets.to(dev))
    for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        if b > a:
            ref, tol = product(values(x[a:b]), w, e)
            check(y[a:b], ref, rounded(ref, tol, dtype))
    assert (y[-3:] == 0).all()


def test_the_most_tokens_of_a_layer():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    tokens, hidden, inter, experts, top_k, dtype = 65535, 64, 32, 20, 16, "bf16"     # 2^20 - 16 pairs
    gate, up = (stack(inter, hidden, 32, 4, dtype, experts, s, dev) for s in (1, 500))
    down = stack(hidden, inter, 32, 4, dtype, experts, 900, dev)
    x = synth.normal_x((tokens, hidden), dtype, seed=1)
    router = synth.normal_x((tokens, experts), dtype, seed=2)
    y = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, top_k)
    ref, tol = reference(x, router, gate, up, down, top_k, True, dtype)
    check(y, ref, tol)


def test_page_work_in_a_replayed_graph():
    """Fork, page copies and a move to other pages, captured once and replayed on new data, between
    eager work; and the same on another stream."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    pages, batch, blocks, page, rows, new, heads, dim = 300, 4, 6, 16, 12, 8, 2, 64
    cache = q.kv_cache(pages, page, heads, dim, 32, "bf16", dev)
    every = torch.arange(pages * page, dtype=torch.int32, device=dev)
    k, v = (_rows((pages * page, heads, dim), "bf16", s).to(dev) for s in (1, 2))
    refs, work = (torch.zeros(pages, dtype=torch.int32, device=dev) for _ in range(2))
    table = torch.zeros(batch, blocks, dtype=torch.int32, device=dev)
    lengths, start = (torch.zeros(batch, dtype=torch.int32, device=dev) for _ in range(2))
    parents, want = (torch.zeros(rows, dtype=torch.int32, device=dev) for _ in range(2))
    to = torch.zeros(batch, 1, dtype=torch.int32, device=dev)
    index = torch.zeros(batch, page, dtype=torch.int32, device=dev)

    def step():
        q.kv_append(cache, k, v, every)
        work.copy_(refs)
        out = q.kv_fork(work, table, lengths, parents, page, want, blocks=new)
        q.kv_copy_pages(cache, out[1], out[2])
        q.kv_move(cache, table, index, start, to_table=to)
        return (*out, *q.kv_read(cache, every))

    def fill(seed):
        r, t, n, p, w = cut_inputs(seed, pages - batch, batch, blocks, page, rows, 30)
        g = np.random.RandomState(seed)
        r = r + [1] * batch                              # the pages that are moved to are held too
        for d, s in ((refs, r), (table, t), (lengths, n), (parents, p), (want, w),
                     (to, [[pages - 1 - b] for b in range(batch)]), (start, g.randint(0, 3, batch).tolist()),
                     (index, [g.randint(-1, m, page).tolist() for m in n])):
            d.copy_(torch.tensor(s, dtype=torch.int32))
        return fork_rule(r, t, n, p, page, w, new)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (10, 20, 30, 40):
        expected = fill(seed)
        eager = [t.clone() for t in step()]
        graph.replay()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
        assert (held[0].tolist(), work.tolist(), held[1].tolist(), held[2].tolist(), held[3].item()) == expected
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step()
        side.synchronize()
        for a, b in zip(other, eager):
            assert torch.equal(a, b)
