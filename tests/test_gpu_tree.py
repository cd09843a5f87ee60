"""Drafted trees over the 4-bit cache: masks, attention, acceptance, moves, and the page work of
forks, against references written from the definitions."""
import numpy as np
import pytest
import torch

from qmm_testlib import TORCH_DTYPE, half_bits, require_gpu, values
from test_gpu_kv_cache import Setup, _rows
from tree_testlib import accept_reference, fork_reference, masked_reference, path_up, random_parents, seen_by

pytestmark = pytest.mark.gpu


def _ints(rows, dev):
    return torch.tensor(rows, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- masks

@pytest.mark.parametrize("batch,nodes,window", [(1, 1, 0), (3, 31, 0), (2, 32, 2), (5, 33, 1), (2, 200, 0), (1, 1024, 5),
                                                (1, 1024, 0)])
def test_tree_mask(batch, nodes, window):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    parents = random_parents(batch, nodes, nodes + window, drop=0.1)
    wide = torch.full((batch, nodes + 3), 7, dtype=torch.int32)
    wide[:, :nodes] = parents
    mask, depth = q.tree_mask(wide.to(dev)[:, :nodes], window=window)
    bits = mask.cpu().numpy().view(np.uint32)
    assert bits.shape == (batch, nodes, (nodes + 31) // 32)
    for b in range(batch):
        row = parents[b].tolist()
        for i in range(nodes):
            path = path_up(row, i)
            want = sorted(path[:window] if window else path)
            got = [j for j in range(32 * bits.shape[2]) if (int(bits[b, i, j // 32]) >> (j % 32)) & 1]
            assert got == want, (b, i)
            assert depth[b, i].item() == max(0, len(path) - 1)


def test_tree_mask_of_a_chain_is_causal():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    chain = torch.arange(-1, 1023, dtype=torch.int32, device=dev)[None]
    mask, depth = q.tree_mask(chain)
    assert torch.equal(depth[0], torch.arange(1024, dtype=torch.int32, device=dev))
    bits = np.unpackbits(mask[0].cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    assert np.array_equal(bits, np.tril(np.ones((1024, 1024), np.uint8)))


# ---------------------------------------------------------------- attention

TREES = [
    # lengths, nodes, heads, rep, dim, group, page, window, dtype
    ([1, 2, 33, 300], 1, 2, 4, 128, 64, 16, 0, "bf16"),              # a tree of its root
    ([0, 13, 14, 45, 509], 13, 2, 4, 128, 64, 16, 0, "bf16"),        # no tokens, no context
    ([7, 100], 7, 1, 1, 64, 32, 48, 0, "fp16"),
    ([70, 250], 33, 3, 2, 64, 64, 32, 0, "bf16"),
    ([64, 1025], 64, 1, 3, 128, 32, 16, 0, "bf16"),
    ([2500], 20, 1, 8, 128, 128, 256, 0, "fp16"),
    ([90, 400], 40, 1, 2, 256, 64, 16, 0, "bf16"),
    ([90, 200], 31, 2, 4, 256, 32, 32, 0, "fp16"),
    ([50, 333], 50, 1, 4, 64, 32, 16, 37, "fp16"),                   # a window that starts in the context
    ([100, 999], 30, 2, 2, 128, 64, 16, 3, "bf16"),                  # one that starts in the tree, mostly
    ([40, 500], 20, 1, 2, 128, 128, 16, 1, "bf16"),                  # a window of the node itself
    ([64, 200, 0], 64, 2, 4, 128, 64, 64, 0, "bf16"),                # 256 rows: two tiles of 16 per wave
    ([211, 330], 211, 1, 3, 128, 32, 48, 0, "fp16"),
    ([130, 600], 130, 1, 2, 128, 128, 16, 100, "bf16"),
    ([256, 400], 256, 1, 4, 64, 64, 16, 0, "fp16"),
    ([150, 260], 150, 1, 8, 256, 32, 32, 0, "bf16"),
    ([1024, 1100], 1024, 1, 1, 64, 32, 16, 40, "bf16"),              # the largest tree
]


@pytest.mark.parametrize("lengths,nodes,heads,rep,dim,group,page,window,dtype", TREES)
def test_attend_tree_matches_float64(lengths, nodes, heads, rep, dim, group, page, window, dtype):
    import bit_affine_quantized_qmv_amd as q
    s = Setup(lengths, heads, dim, group, page, dtype, seed=dim + nodes)
    dev = s.len_dev.device
    parents = random_parents(len(lengths), nodes, nodes, drop=0.02)
    mask, depth = q.tree_mask(parents.to(dev), window=window)
    queries = _rows((len(lengths), nodes, heads * rep, dim), dtype, 77, loud=False)
    y = q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask, depth, window=window)
    again = q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask, depth, window=window,
                             max_length=max(lengths))
    prompt = nodes * rep >= (256 if dim == 128 else 1024)
    for got in (values(y), values(again)):
        assert np.isfinite(got).all()
        for b, n in enumerate(lengths):
            see = seen_by(parents[b].tolist(), n, window) if n else np.zeros((nodes, 0), bool)
            ref, tol = masked_reference(queries[b], s.k[b], s.v[b], see, group, dtype, dim ** -0.5, prompt)
            err = np.abs(got[b] - ref)
            assert (err <= tol).all(), "sequence %d (%d tokens): worst %.3g of the bound" % (
                b, n, (err / np.maximum(tol, 1e-30)).max())


def test_attend_tree_of_a_chain_is_the_draft_form():
    import bit_affine_quantized_qmv_amd as q
    for nodes, rep, dim, window in ((9, 2, 128, 0), (80, 4, 128, 0), (30, 4, 64, 11)):
        s = Setup([nodes, 333], 2, dim, 32, 16, "bf16", seed=4)
        dev = s.len_dev.device
        chain = torch.arange(-1, nodes - 1, dtype=torch.int32, device=dev).expand(2, nodes).contiguous()
        mask, depth = q.tree_mask(chain, window=window)
        queries = _rows((2, nodes, 2 * rep, dim), "bf16", 5, loud=False).to(dev)
        y = q.kv_attend_tree(queries, s.cache, s.table, s.len_dev, mask, depth, window=window)
        want = q.kv_attend(queries, s.cache, s.table, s.len_dev, window=window)
        # one step of bf16, and 2^-14 of the largest |v| (below 32) for the operands of the second product
        assert torch.allclose(y.float(), want.float(), rtol=2 ** -7, atol=2 ** -9)


def test_attend_tree_lengths_pages_and_rows_of_nothing():
    """Lengths out of order, pages outside the pool, rows of zeros next to NaN, a caller's own mask."""
    import bit_affine_quantized_qmv_amd as q
    nodes, heads, dim = 20, 2, 128
    for rep in (1, 16):                                  # both forms
        s = Setup([200, 200, 200, 200, 200], heads, dim, 64, 16, "bf16", seed=8)
        dev = s.len_dev.device
        parents = random_parents(5, nodes, 3)
        parents[1, 12:] = -2                             # a smaller tree: its last page is nobody's
        mask, depth = q.tree_mask(parents.to(dev))
        table = s.table.clone()
        table[1, 12] = -1                                # tokens 192 .. 199 of sequence 1: padding, not seen
        table[2, 12] = s.cache.pages                     # those of sequence 2 are seen
        lengths = s.len_dev.clone()
        lengths[3], lengths[4] = nodes - 1, 209          # too short for the tree, longer than max_length
        queries = _rows((5, nodes, heads * rep, dim), "bf16", 6, loud=False)
        y = q.kv_attend_tree(queries.to(dev), s.cache, table, lengths, mask, max_length=208)
        got = values(y)
        assert np.isnan(got[3:]).all()
        assert (got[1, 12:] == 0).all() and np.isfinite(got[:2]).all()
        for i in range(nodes):                           # a node of sequence 2 that sees one from 192 on
            lost = any(180 + u >= 192 for u in path_up(parents[2].tolist(), i))
            assert np.isnan(got[2, i]).all() if lost else np.isfinite(got[2, i]).all(), i
        for b in range(2):
            ref, tol = masked_reference(queries[b], s.k[b], s.v[b], seen_by(parents[b].tolist(), 200, 0), 64, "bf16",
                                        dim ** -0.5, rep == 16)
            assert (np.abs(got[b] - ref) <= tol).all()
        # any mask: every node sees every node, but one that sees nothing
        own = torch.full((5, nodes, 1), 2 ** nodes - 1, dtype=torch.int32, device=dev)
        own[:, 5] = 0
        y = q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, own)
        see = np.ones((nodes, 200), bool)
        see[5] = False
        for b in range(5):
            ref, tol = masked_reference(queries[b], s.k[b], s.v[b], see, 64, "bf16", dim ** -0.5, rep == 16)
            assert (np.abs(values(y)[b] - ref) <= tol).all()


def test_attend_tree_unseen_nodes_that_are_not_finite():
    import bit_affine_quantized_qmv_amd as q
    nodes, dim = 18, 128
    for rep in (2, 16):
        s = Setup([100], 1, dim, 64, 16, "bf16", seed=12)
        dev = s.len_dev.device
        parents = torch.full((1, nodes), 0, dtype=torch.int32)
        parents[0, 0] = -1
        parents[0, 9] = -2                               # no node: its rows are what they were before, NaN
        slot = s.slots[82 + 9:82 + 10]
        bad = torch.full((1, 1, dim), float("nan"), dtype=torch.bfloat16, device=dev)
        side = s.cache.data.clone()
        q.kv_append(s.cache, bad, bad, slot)
        mask, _ = q.tree_mask(parents.to(dev))
        queries = _rows((1, nodes, rep, dim), "bf16", 6, loud=False)
        y = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask))
        s.cache.data.copy_(side)
        ref, tol = masked_reference(queries[0], s.k[0], s.v[0], seen_by(parents[0].tolist(), 100, 0), 64, "bf16",
                                    dim ** -0.5, nodes * rep >= 256)
        assert (np.abs(y[0] - ref) <= tol).all() and (y[0, 9] == 0).all()


def test_attend_tree_nodes_that_are_not_finite_reach_their_descendants_only():
    import bit_affine_quantized_qmv_amd as q
    nodes, dim = 34, 128
    for rep, group in ((2, 64), (8, 64), (16, 128)):     # one tile of 16 rows per wave, and two
        s = Setup([120], 1, dim, group, 16, "bf16", seed=14)
        dev = s.len_dev.device
        parents = random_parents(1, nodes, 21)
        row = parents[0].tolist()
        lost = next(i for i in range(3, nodes) if sum(i in path_up(row, j) for j in range(nodes)) >= 3)
        bad = torch.full((1, 1, dim), float("inf"), dtype=torch.bfloat16, device=dev)
        q.kv_append(s.cache, bad, bad, s.slots[120 - nodes + lost:120 - nodes + lost + 1])
        mask, _ = q.tree_mask(parents.to(dev))
        queries = _rows((1, nodes, rep, dim), "bf16", 6, loud=False)
        y = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask))[0]
        ref, tol = masked_reference(queries[0], s.k[0], s.v[0], seen_by(row, 120, 0), group, "bf16", dim ** -0.5,
                                    nodes * rep >= 256)
        for i in range(nodes):
            if lost in path_up(row, i):
                assert np.isnan(y[i]).all(), i
            else:
                assert (np.abs(y[i] - ref[i]) <= tol[i]).all(), i


def test_attend_tree_of_many_sequences_in_any_order_of_lengths():
    import bit_affine_quantized_qmv_amd as q
    nodes, heads, rep, dim = 5, 1, 2, 64
    for batch in (64, 65, 130):
        lengths = [(0 if i % 9 == 4 else nodes + (37 * i) % 61) for i in range(batch)]
        s = Setup(lengths, heads, dim, 32, 16, "bf16", seed=batch)
        dev = s.len_dev.device
        parents = random_parents(batch, nodes, 3)
        mask, depth = q.tree_mask(parents.to(dev))
        queries = _rows((batch, nodes, heads * rep, dim), "bf16", 6, loud=False).to(dev)
        y = q.kv_attend_tree(queries, s.cache, s.table, s.len_dev, mask, depth)
        for b in range(batch):
            one = q.kv_attend_tree(queries[b:b + 1], s.cache, s.table[b:b + 1], s.len_dev[b:b + 1], mask[b:b + 1])
            assert torch.equal(one[0], y[b]), b


def test_attend_tree_strides_workspace_and_stream():
    import bit_affine_quantized_qmv_amd as q
    nodes, heads, rep, dim = 24, 2, 2, 64
    s = Setup([60, 24, 3000], heads, dim, 32, 16, "fp16", seed=2)
    dev = s.len_dev.device
    parents = random_parents(3, nodes, 9)
    mask, depth = q.tree_mask(parents.to(dev))
    big = _rows((heads * rep + 2, 3, nodes, dim + 8), "fp16", 6, loud=False).to(dev)
    view = big[1:-1, :, :, :dim].permute(1, 2, 0, 3)
    want = q.kv_attend_tree(view.contiguous(), s.cache, s.table, s.len_dev, mask)
    ws = q.kv_attend_tree_workspace(view, s.cache, 3008)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.kv_attend_tree(view, s.cache, s.table, s.len_dev, mask, depth, out=out, workspace=ws, max_length=3008)
    side.synchronize()
    assert torch.equal(out, q.kv_attend_tree(view, s.cache, s.table, s.len_dev, mask, max_length=3008))


# ---------------------------------------------------------------- acceptance

@pytest.mark.parametrize("batch,nodes", [(1, 1), (3, 13), (64, 63), (2, 65), (2, 1024)])
def test_tree_accept(batch, nodes):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    g = np.random.RandomState(nodes)
    parents = random_parents(batch, nodes, nodes, drop=0.02)
    if batch > 2:
        parents[2, 0] = -2
    tokens, sampled = (torch.from_numpy(g.randint(0, 3, (batch, nodes + 2)).astype(np.int32)) for _ in range(2))
    path, count, last = q.tree_accept(parents.to(dev), tokens.to(dev)[:, :nodes], sampled.to(dev)[:, 1:-1])
    for b in range(batch):
        want, end = accept_reference(parents[b].tolist(), tokens[b, :nodes].tolist(), sampled[b, 1:-1].tolist())
        assert path[b].tolist() == want + [-1] * (nodes - len(want))
        assert count[b].item() == len(want) and last[b].item() == end


def test_tree_accept_of_a_long_chain():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    chain = torch.arange(-1, 1023, dtype=torch.int32, device=dev)[None]
    tokens = torch.zeros(1, 1024, dtype=torch.int32, device=dev)
    sampled = tokens.clone()
    sampled[0, 1000] = 9
    path, count, last = q.tree_accept(chain, tokens, sampled)
    assert path[0, :1001].tolist() == list(range(1001)) and count.item() == 1001 and last.item() == 9


# ---------------------------------------------------------------- moves

def _all_slots(cache, dev):
    return torch.arange(cache.pages * cache.page_size, dtype=torch.int32, device=dev)


def _bits(cache, dev):
    """Every row of the cache as bit patterns [slot, heads, 2 * dim]."""
    import bit_affine_quantized_qmv_amd as q
    k, v = q.kv_read(cache, _all_slots(cache, dev))
    return np.concatenate([half_bits(k), half_bits(v)], -1)


def _filled(pages, page, heads, dim, group, dtype, seed):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    cache = q.kv_cache(pages, page, heads, dim, group, dtype, dev)
    n = pages * page
    q.kv_append(cache, _rows((n, heads, dim), dtype, seed).to(dev), _rows((n, heads, dim), dtype, seed + 1).to(dev),
                _all_slots(cache, dev))
    return cache, dev


MOVES = [
    # dim, group, page, heads, dtype, blocks, in place
    (64, 32, 16, 3, "bf16", 9, True), (64, 64, 48, 1, "fp16", 4, True), (128, 32, 16, 2, "fp16", 20, True),
    (128, 64, 64, 1, "bf16", 5, True), (256, 128, 32, 2, "bf16", 6, True), (256, 32, 16, 1, "fp16", 9, True),
    (64, 32, 16, 2, "fp16", 9, False), (128, 128, 80, 2, "bf16", 3, False), (256, 64, 16, 1, "bf16", 12, False),
]


@pytest.mark.parametrize("dim,group,page,heads,dtype,blocks,in_place", MOVES)
def test_move(dim, group, page, heads, dtype, blocks, in_place):
    import bit_affine_quantized_qmv_amd as q
    batch = 4
    cache, dev = _filled(2 * batch * blocks + 3, page, heads, dim, group, dtype, dim + page)
    g = np.random.RandomState(dim + group + page)
    perm = g.permutation(cache.pages)[:2 * batch * blocks].reshape(2, batch, blocks)
    table, to = perm[0].copy(), perm[0] if in_place else perm[1].copy()
    length = blocks * page
    count = length - 5
    index, start, origin = np.full((batch, count + 1), -1), np.zeros(batch, int), np.zeros(batch, int)
    for n in range(batch):
        start[n] = [0, 3, page + 1, 7][n]
        if in_place:
            origin[n] = start[n]
            room = length - start[n]
            kept = np.sort(g.permutation(room)[:[room // 3, room - 9, 40, 1][n]])
            kept = kept[:count + 1]
            index[n, :len(kept)] = kept
            index[n, len(kept) // 2] = -1 if n == 1 else index[n, len(kept) // 2]   # a hole
        else:
            origin[n] = [0, 5, 2, 0][n]
            m = [count, 100, 33, 1][n]
            m = min(m, length - start[n])
            index[n, :m] = g.randint(-1, length - origin[n], m)                     # any order, some twice
    before = _bits(cache, dev)
    want = before.copy()
    slot = lambda t, n, p: t[n, p // page] * page + p % page  # noqa: E731
    for n in range(batch):
        for i, x in enumerate(index[n]):
            if x >= 0 and start[n] + i < length:
                want[slot(to, n, start[n] + i)] = before[slot(table, n, origin[n] + x)]
    wide = torch.zeros(batch, blocks + 2, dtype=torch.int32, device=dev)
    wide[:, 1:-1] = torch.from_numpy(table).to(dev)
    q.kv_move(cache, wide[:, 1:-1], _ints(index.tolist(), dev), _ints(start.tolist(), dev), _ints(origin.tolist(), dev),
              None if in_place else _ints(to.tolist(), dev))
    assert np.array_equal(_bits(cache, dev), want)


def test_move_skips_positions_without_a_page():
    import bit_affine_quantized_qmv_amd as q
    cache, dev = _filled(6, 16, 2, 64, 32, "bf16", 1)
    before = _bits(cache, dev)
    table = _ints([[2, -1, 6, 4]], dev)
    index = _ints([[3, 17, 40, 63, 64, 2 ** 31 - 1, -2 ** 31, 50]], dev)
    to = _ints([[1]], dev)
    q.kv_move(cache, table, index, _ints([10], dev), to_table=to)     # positions 10 .. 15 have a page, 16 and 17 none
    want = before.copy()
    want[16 + 10], want[16 + 13] = before[2 * 16 + 3], before[4 * 16 + 15]
    assert np.array_equal(_bits(cache, dev), want)
    q.kv_move(cache, table, index[:, :0], _ints([10], dev))
    q.kv_move(cache, table[:0], index[:0], _ints([0], dev)[:0])
    q.kv_move(cache, table, index, _ints([2 ** 31 - 4], dev))
    q.kv_move(cache, table, index, _ints([-3], dev), to_table=to)     # positions -3 .. 4
    want[16 + 0] = before[4 * 16 + 15]
    want[16 + 4] = before[4 * 16 + 2]
    assert np.array_equal(_bits(cache, dev), want)


def test_copy_pages():
    import bit_affine_quantized_qmv_amd as q
    for dim, group, page, heads in ((64, 32, 16, 1), (128, 64, 48, 5), (256, 128, 128, 3)):
        cache, dev = _filled(9, page, heads, dim, group, "bf16", dim)
        before = cache.data.clone()
        src, dst = [4, -1, 3, 4, 9, 2, 0], [0, 1, -1, 8, 2, 10 ** 9, 7]
        src[6] = 5
        q.kv_copy_pages(cache, _ints(src, dev), _ints(dst, dev))
        want = before.clone()
        want[0], want[8], want[7] = before[4], before[4], before[5]
        assert torch.equal(cache.data, want)
        q.kv_copy_pages(cache, _ints(src, dev)[:0], _ints(dst, dev)[:0])


# ---------------------------------------------------------------- forks

def _pool(pages, batch, blocks, page, seed, shared=False):
    """refs, table and lengths of `batch` sequences; some entries past the length, some shared."""
    g = np.random.RandomState(seed)
    free = list(g.permutation(pages))
    table, lengths = [], []
    for n in range(batch):
        length = int(g.randint(0, blocks * page + 1))
        held = min(blocks, -(-length // page) + int(g.randint(0, 2)))
        row = [int(free.pop()) for _ in range(held)]
        if shared and n and held and len(table[n - 1]) and table[n - 1][0] >= 0:
            k = min(held, sum(p >= 0 for p in table[n - 1]), int(g.randint(0, blocks + 1)))
            row[:k] = table[n - 1][:k]
        table.append(row + [-1] * (blocks - held))
        lengths.append(length)
    refs = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    return refs, table, lengths


FORKS = [
    # pages, batch, blocks, page, rows, new blocks, want, shared
    (64, 4, 5, 16, 4, 5, "same", False),
    (300, 8, 6, 16, 32, 9, "grow", False),
    (300, 8, 6, 48, 20, 9, "any", True),
    (60, 8, 6, 16, 32, 9, "grow", False),          # not enough pages
    (9000, 40, 300, 16, 70, 310, "any", True),     # several segments of the pool, rows wider than a workgroup
    (40, 1, 3, 16, 1, 2, "grow", False),           # a new table that is too narrow
    (40, 3, 4, 16, 0, 4, "same", True),            # everything ends
    (40, 0, 4, 16, 3, 4, "any", False),            # everything begins
    (5000, 300, 4, 64, 400, 4, "same", True),
]


@pytest.mark.parametrize("pages,batch,blocks,page,rows,new,how,shared", FORKS)
def test_fork(pages, batch, blocks, page, rows, new, how, shared):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    g = np.random.RandomState(pages + rows)
    refs, table, lengths = _pool(pages, batch, blocks, page, pages, shared)
    for step in range(3):
        parents = g.randint(-1, batch + 1, rows).tolist()
        if how == "same":
            want = None
        else:
            base = [lengths[p] if 0 <= p < batch else 0 for p in parents]
            want = [max(-1, b + int(g.randint(0 if how == "grow" else -2 * page, 2 * page))) for b in base]
        out, after, src, dst, short = fork_reference(refs, table, lengths, parents, page, want, new)
        d_refs = _ints(refs, dev)
        got = q.kv_fork(d_refs, _ints(table, dev).reshape(batch, blocks), _ints(lengths, dev), _ints(parents, dev), page,
                        None if want is None else _ints(want, dev), blocks=new)
        assert got[0].tolist() == out and d_refs.tolist() == after
        assert (got[1].tolist(), got[2].tolist(), got[3].item()) == (src, dst, short)
        assert min(after) >= 0
        # go on from there
        lengths = [min(n, new * page) for n in (want if want is not None else
                                                [lengths[p] if 0 <= p < batch else 0 for p in parents])]
        refs, table, batch, blocks = after, out, rows, new


def test_fork_keeps_pages_that_it_copies_from():
    """Two rows cut back into a page that both hold: each gets a copy, and the page itself is free
    only after the call."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    refs = _ints([0, 2, 2, 0], dev)
    table, src, dst, short = q.kv_fork(refs, _ints([[2, 1], [2, 1]], dev), _ints([20, 32], dev), _ints([0, 1], dev), 16,
                                       _ints([20, 25], dev))
    assert table.tolist() == [[2, 0], [2, 3]] and src.tolist() == [1, 1] and dst.tolist() == [0, 3]
    assert short.item() == 0 and refs.tolist() == [1, 0, 2, 1]


# ---------------------------------------------------------------- a step of all of them, in a graph

def test_accepted_path_in_a_replayed_graph():
    """Append, mask, attention, acceptance and move, captured once and replayed on new data."""
    import bit_affine_quantized_qmv_amd as q
    nodes, heads, rep, dim, group, page, dtype = 21, 2, 2, 64, 32, 16, "bf16"
    context = [5, 50, 130]
    s = Setup([c + nodes for c in context], heads, dim, group, page, dtype, seed=3)
    dev = s.len_dev.device
    n_slots = torch.stack([s.slots[sum(c + nodes for c in context[:b]) + context[b]:][:nodes] for b in range(3)])
    start = _ints(context, dev)
    parents, tokens, sampled = (torch.zeros(3, nodes, dtype=torch.int32, device=dev) for _ in range(3))
    k, v = (torch.zeros(3 * nodes, heads, dim, dtype=TORCH_DTYPE[dtype], device=dev) for _ in range(2))
    queries = torch.zeros(3, nodes, heads * rep, dim, dtype=TORCH_DTYPE[dtype], device=dev)
    flat = n_slots.flatten().contiguous()

    def step():
        q.kv_append(s.cache, k, v, flat)
        mask, depth = q.tree_mask(parents)
        y = q.kv_attend_tree(queries, s.cache, s.table, s.len_dev, mask, depth)
        path, count, last = q.tree_accept(parents, tokens, sampled)
        q.kv_move(s.cache, s.table, path, start, origin=start)
        return (y, path, count, last) + q.kv_read(s.cache, flat)

    def fill(seed):
        g = np.random.RandomState(seed)
        p = random_parents(3, nodes, seed)
        p[:, 0] = -1
        parents.copy_(p)
        for t in (tokens, sampled):
            t.copy_(torch.from_numpy(g.randint(0, 2, (3, nodes)).astype(np.int32)))
        for i, t in enumerate((k, v, queries)):
            t.copy_(_rows(tuple(t.shape), dtype, seed + i, loud=i < 2))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (10, 20, 30):
        fill(seed)
        eager = [t.clone() for t in step()]
        graph.replay()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
        for b, c in enumerate(context):
            see = seen_by(parents[b].tolist(), c + nodes, 0)
            mine = slice(b * nodes, (b + 1) * nodes)
            kk, vv = torch.cat([s.k[b][:c], k[mine].cpu()]), torch.cat([s.v[b][:c], v[mine].cpu()])
            ref, tol = masked_reference(queries[b].cpu(), kk, vv, see, group, dtype, dim ** -0.5, False)
            assert (np.abs(values(held[0][b]) - ref) <= tol).all()
            path, last = accept_reference(parents[b].tolist(), tokens[b].tolist(), sampled[b].tolist())
            assert held[2][b].item() == len(path) and held[3][b].item() == last
            order = path + list(range(len(path), nodes))
            other = q.kv_cache(4, 16, heads, dim, group, dtype, dev)
            slots = torch.arange(nodes, dtype=torch.int32, device=dev)
            q.kv_append(other, k[mine][order], v[mine][order], slots)
            for got, want in zip(held[4:], q.kv_read(other, slots)):
                assert torch.equal(got[mine], want)


def test_beams_over_forked_pages():
    """Steps of a beam search: fork, page copies, append, attention, each against a cache of its own."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    heads, rep, dim, group, page, dtype, pages = 2, 2, 64, 32, 16, "bf16", 40
    g = np.random.RandomState(5)
    text = [13, 31, 16]                                  # tokens of the sequences at first
    rows = [[[_rows((1, heads, dim), dtype, 1000 * b + 2 * j + side) for side in (0, 1)] for j in range(n)]
            for b, n in enumerate(text)]
    cache = q.kv_cache(pages, page, heads, dim, group, dtype, dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[7] = 1                                          # a page of somebody else's
    table, _, _, short = q.kv_fork(refs, _ints([[]] * 0, dev).reshape(0, 8), _ints([], dev), _ints([-1] * 3, dev), page,
                                   _ints(text, dev), blocks=8)
    at = table.cpu().numpy()
    slots = [at[b, j // page] * page + j % page for b, n in enumerate(text) for j in range(n)]
    q.kv_append(cache, *(torch.cat([r[side] for b in rows for r in b]).to(dev) for side in (0, 1)), _ints(slots, dev))
    assert short.item() == 0
    for step in range(5):
        n = [4, 6, 2, 6, 5][step]
        parents = g.randint(0, len(rows), n).tolist()
        lengths = [len(r) for r in rows]
        want = [lengths[p] + 1 for p in parents]
        table, src, dst, short = q.kv_fork(refs, table, _ints(lengths, dev), _ints(parents, dev), page, _ints(want, dev))
        q.kv_copy_pages(cache, src, dst)
        assert short.item() == 0
        new = [[_rows((1, heads, dim), dtype, 50000 + 100 * step + 2 * b + side) for side in (0, 1)] for b in range(n)]
        rows = [rows[p] + [new[b]] for b, p in enumerate(parents)]
        at = table.cpu().numpy()
        last = _ints([at[b, (m - 1) // page] * page + (m - 1) % page for b, m in enumerate(want)], dev)
        q.kv_append(cache, *(torch.cat([r[side] for r in new]).to(dev) for side in (0, 1)), last)
        # the same beams, each in pages of its own
        own = q.kv_cache(8 * n, page, heads, dim, group, dtype, dev)
        own_table = torch.arange(8 * n, dtype=torch.int32, device=dev).reshape(n, 8)
        own_slots = _ints([b * 8 * page + j for b, m in enumerate(want) for j in range(m)], dev)
        q.kv_append(own, *(torch.cat([r[side] for b in rows for r in b]).to(dev) for side in (0, 1)), own_slots)
        slots = _ints([at[b, j // page] * page + j % page for b, m in enumerate(want) for j in range(m)], dev)
        for x, y in zip(q.kv_read(cache, slots), q.kv_read(own, own_slots)):
            assert torch.equal(x, y)
        queries = _rows((n, 1, heads * rep, dim), dtype, 900 + step, loud=False).to(dev)
        assert torch.equal(q.kv_attend(queries, cache, table, _ints(want, dev), max_length=128),
                           q.kv_attend(queries, own, own_table, _ints(want, dev), max_length=128))
        # every page is counted as often as the table names it
        count = np.bincount(at[at >= 0].ravel(), minlength=pages)
        count[7] += 1
        assert refs.tolist() == count.tolist()
