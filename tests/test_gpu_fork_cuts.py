"""Forks whose rows keep different parts of one sequence: against the definition, entry by entry, and
as beams that go on writing, each against a cache of its own."""
import numpy as np
import pytest
import torch

from fork_testlib import cut_inputs, fork_rule, kept_tokens, shared_writes
from qmm_testlib import require_gpu
from test_gpu_kv_cache import _rows
from test_gpu_tree import FORKS, _ints, _pool

pytestmark = pytest.mark.gpu


def fork(refs, table, lengths, parents, page, want, blocks):
    """kv_fork's results as fork_rule's."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    d_refs = _ints(refs, dev)
    width = len(table[0]) if table else 0
    got = q.kv_fork(d_refs, _ints(table, dev).reshape(len(table), width), _ints(lengths, dev), _ints(parents, dev), page,
                    None if want is None else _ints(want, dev), blocks=blocks)
    return got[0].tolist(), d_refs.tolist(), got[1].tolist(), got[2].tolist(), got[3].item()


CUTS = [
    # pages, batch, blocks, page, rows, new blocks, spread
    (8, 1, 4, 16, 2, 4, 20), (200, 4, 6, 16, 12, 8, 30), (200, 1, 6, 48, 40, 8, 30), (4000, 3, 6, 16, 700, 8, 60),
    (9000, 20, 300, 16, 70, 310, 200), (60, 4, 6, 16, 30, 8, 30),
]


@pytest.mark.parametrize("pages,batch,blocks,page,rows,new,spread", CUTS)
@pytest.mark.parametrize("from_start", [True, False])
def test_fork_of_rows_that_keep_different_parts(pages, batch, blocks, page, rows, new, spread, from_start):
    for seed in range(5):
        refs, table, lengths, parents, want = cut_inputs(seed, pages, batch, blocks, page, rows, spread, from_start)
        got = fork(refs, table, lengths, parents, page, want, new)
        assert got == fork_rule(refs, table, lengths, parents, page, want, new), seed
        assert not shared_writes(got[0], got[1], lengths, parents, page, want)


@pytest.mark.parametrize("pages,batch,blocks,page,rows,new,how,shared", FORKS)
def test_fork_of_shared_pools(pages, batch, blocks, page, rows, new, how, shared):
    """The pools of test_fork, step after step."""
    g = np.random.RandomState(pages + rows)
    refs, table, lengths = _pool(pages, batch, blocks, page, pages, shared)
    for step in range(3):
        parents = g.randint(-1, len(table) + 1, rows).tolist()
        want = None
        if how != "same":
            base = [lengths[p] if 0 <= p < len(table) else 0 for p in parents]
            want = [max(-1, b + int(g.randint(0 if how == "grow" else -2 * page, 2 * page))) for b in base]
        got = fork(refs, table, lengths, parents, page, want, new)
        assert got == fork_rule(refs, table, lengths, parents, page, want, new)
        assert not shared_writes(got[0], got[1], lengths, parents, page, want)
        lengths = [min(w, new * page) for _, w, _ in kept_tokens(lengths, parents, want)]
        table, refs = got[:2]


def test_beams_cut_back_over_forked_pages():
    """Beams that fall back to different lengths of one text and go on: fork, page copies, append,
    then rows and attention against caches of their own."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    heads, rep, dim, group, page, dtype, pages, width = 2, 2, 64, 32, 16, "bf16", 60, 8
    g = np.random.RandomState(11)
    made = iter(range(10 ** 6))

    def token():
        n = next(made)
        return [_rows((1, heads, dim), dtype, 2 * n + side) for side in (0, 1)]

    rows = [[token() for _ in range(n)] for n in (56, 31)]
    cache = q.kv_cache(pages, page, heads, dim, group, dtype, dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    table, _, _, short = q.kv_fork(refs, torch.zeros(0, width, dtype=torch.int32, device=dev), _ints([], dev),
                                   _ints([-1, -1], dev), page, _ints([len(r) for r in rows], dev))

    def append(c, t, who, first):
        """Tokens first[b] .. of every beam into its pages."""
        at = t.cpu().numpy()
        slots = [at[b, j // page] * page + j % page for b, r in enumerate(who) for j in range(first[b], len(r))]
        new = [x for b, r in enumerate(who) for x in r[first[b]:]]
        q.kv_append(c, *(torch.cat([x[side] for x in new]).to(dev) for side in (0, 1)), _ints(slots, dev))

    append(cache, table, rows, [0, 0])
    for step in range(6):
        parents = ([0, 0, 1, 0, 0] if step == 0 else g.randint(0, len(rows), 5).tolist())
        lengths = [len(r) for r in rows]
        keep = [20, 56, 31, 33, 48] if step == 0 else [int(g.randint(lengths[p] // 2, lengths[p] + 1)) for p in parents]
        # a beam that keeps everything asks for the room of the token that it adds, the others have it in
        # the block that they keep in part
        want = [k + 1 if k == lengths[p] or k % page == 0 else k for k, p in zip(keep, parents)]
        keep = [min(w, lengths[p]) for w, p in zip(want, parents)]
        table, src, dst, short = q.kv_fork(refs, table, _ints(lengths, dev), _ints(parents, dev), page, _ints(want, dev))
        q.kv_copy_pages(cache, src, dst)
        assert short.item() == 0
        rows = [rows[p][:k] for p, k in zip(parents, keep)]
        grown = [len(r) for r in rows]
        rows = [r + [token()] if len(r) % page or w > len(r) else r for r, w in zip(rows, want)]
        append(cache, table, rows, grown)
        own = q.kv_cache(width * len(rows), page, heads, dim, group, dtype, dev)
        own_table = torch.arange(width * len(rows), dtype=torch.int32, device=dev).reshape(len(rows), width)
        append(own, own_table, rows, [0] * len(rows))
        at = table.cpu().numpy()
        slots = [[t[j // page] * page + j % page for j in range(len(r))] for t, r in zip(at, rows)]
        own_slots = [[b * width * page + j for j in range(len(r))] for b, r in enumerate(rows)]
        for b in range(len(rows)):
            for x, y in zip(q.kv_read(cache, _ints(slots[b], dev)), q.kv_read(own, _ints(own_slots[b], dev))):
                assert torch.equal(x, y), (step, b)
        queries = _rows((len(rows), 1, heads * rep, dim), dtype, 900 + step, loud=False).to(dev)
        now = _ints([len(r) for r in rows], dev)
        assert torch.equal(q.kv_attend(queries, cache, table, now, max_length=width * page),
                           q.kv_attend(queries, own, own_table, now, max_length=width * page))
        assert refs.tolist() == np.bincount(at[at >= 0].ravel(), minlength=pages).tolist()
