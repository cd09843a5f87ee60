"""Every form of tree attention at the edges: pages outside the pool, lengths out of order, masks of the
caller's own, rows of nothing and cached rows that are not finite, each within the bound of the form's
own operands."""
import numpy as np
import pytest
import torch

from qmm_testlib import TORCH_DTYPE, values
from test_gpu_kv_cache import Setup, _rows
from tree_forms import shares_unpacked_values
from tree_testlib import masked_reference, path_up, random_parents, seen_by

pytestmark = pytest.mark.gpu

FORMS = [
    # nodes, query heads per cached head, dim, group, dtype
    (20, 2, 128, 64, "bf16"),           # one tile of 16 rows per wave
    (20, 3, 64, 64, "fp16"),
    (20, 2, 256, 32, "bf16"),
    (20, 16, 128, 64, "bf16"),          # two tiles of 16 rows per wave
    (20, 13, 128, 128, "fp16"),         # (260 rows: the last workgroup's second tile is empty)
    (19, 15, 128, 64, "bf16"),          # (285 rows: a part of it)
    (20, 16, 128, 32, "bf16"),          # values unpacked for many rows: sixteen waves
    (19, 15, 128, 32, "fp16"),
    (20, 52, 64, 32, "bf16"),
    (18, 60, 64, 64, "fp16"),
    (20, 52, 256, 64, "fp16"),          # eight waves
    (20, 52, 256, 128, "bf16"),
]


def bounded(queries, s, b, see, sides=None):
    """masked_reference of sequence b with the bound of the form that the call takes."""
    q_heads, dim = queries.shape[2:]
    heads = s.k[b].shape[1]
    rows = queries.shape[1] * (q_heads // heads)
    k, v = (s.k[b], s.v[b]) if sides is None else sides
    return masked_reference(queries[b], k, v, see, s.group, s.dtype, dim ** -0.5, shares_unpacked_values(rows, dim, s.group))


def within(got, ref, tol):
    err = np.abs(got - ref)
    assert (err <= tol).all(), "worst %.3g of the bound" % (err / np.maximum(tol, 1e-30)).max()


@pytest.mark.parametrize("nodes,rep,dim,group,dtype", FORMS)
def test_within_the_bound_of_its_operands(nodes, rep, dim, group, dtype):
    import bit_affine_quantized_qmv_amd as q
    s = Setup([nodes, 90, 301, 0], 1, dim, group, 16, dtype, seed=nodes + rep)
    dev = s.len_dev.device
    for window in (0, 33):
        parents = random_parents(4, nodes, rep, drop=0.03)
        mask, depth = q.tree_mask(parents.to(dev), window=window)
        queries = _rows((4, nodes, rep, dim), dtype, 9, loud=False)
        for most in (None, 301):
            got = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask, depth, window=window,
                                          max_length=most))
            for b in range(3):
                within(got[b], *bounded(queries, s, b, seen_by(parents[b].tolist(), s.lengths[b], window)))
            assert (got[3] == 0).all()


@pytest.mark.parametrize("nodes,rep,dim,group,dtype", FORMS)
def test_lengths_pages_and_rows_of_nothing(nodes, rep, dim, group, dtype):
    import bit_affine_quantized_qmv_amd as q
    s = Setup([200] * 6, 1, dim, group, 16, dtype, seed=8)
    dev = s.len_dev.device
    parents = random_parents(6, nodes, 3)
    first = 192 - (200 - nodes)                      # the first node of a token from 192 on
    parents[1, first:] = -2                          # a smaller tree
    parents[5] = -2                                  # no tree at all
    mask, depth = q.tree_mask(parents.to(dev))
    last = torch.arange(12, s.table.shape[1])        # blocks of tokens 192 ..
    table = s.table.clone()
    table[1, last] = -1                              # of sequence 1: no node's
    table[2, last] = s.cache.pages                   # of sequence 2: seen
    lengths = s.len_dev.clone()
    lengths[3], lengths[4] = nodes - 1, 209          # too short for the tree, longer than max_length
    queries = _rows((6, nodes, rep, dim), dtype, 6, loud=False)
    got = values(q.kv_attend_tree(queries.to(dev), s.cache, table, lengths, mask, max_length=208))
    assert np.isnan(got[3:5]).all() and (got[5] == 0).all()
    for i in range(nodes):
        lost = any(u >= first for u in path_up(parents[2].tolist(), i))
        assert np.isnan(got[2, i]).all() if lost else np.isfinite(got[2, i]).all(), i
    see = [seen_by(parents[b].tolist(), 200, 0) for b in range(6)]
    for b in (0, 1):
        within(got[b], *bounded(queries, s, b, see[b]))
    assert (got[1, first:] == 0).all()
    # any mask: every node sees every node, but one that sees nothing
    own = torch.full((6, nodes, 1), 2 ** nodes - 1, dtype=torch.int32, device=dev)
    own[:, 5] = 0
    got = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, own))
    all_see = np.ones((nodes, 200), bool)
    all_see[5] = False
    for b in range(6):
        within(got[b], *bounded(queries, s, b, all_see))
    # a page of the context that is nobody's: every row that sees it is lost, the others are not
    table = s.table.clone()
    table[:, 3] = -1
    got = values(q.kv_attend_tree(queries.to(dev), s.cache, table, s.len_dev, own))
    assert np.isnan(np.delete(got, 5, 1)).all() and (got[:, 5] == 0).all()


@pytest.mark.parametrize("nodes,rep,dim,group,dtype", FORMS)
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_nodes_that_are_not_finite_reach_their_descendants_only(nodes, rep, dim, group, dtype, value):
    import bit_affine_quantized_qmv_amd as q
    s = Setup([120, 120, 120], 1, dim, group, 16, dtype, seed=14)
    dev = s.len_dev.device
    parents = random_parents(3, nodes, 21)
    parents[0] = 0
    parents[0, 0] = -1
    parents[0, 9] = -2                               # no node: its row may hold anything
    lost = [9, 4, None]
    rows = [parents[b].tolist() for b in range(3)]
    at = [120 * b + 120 - nodes + lost[b] for b in (0, 1)]
    bad = torch.full((2, 1, dim), float(value), dtype=TORCH_DTYPE[dtype], device=dev)
    fine = torch.cat([s.k[0][:1], s.k[0][:1]]).to(dev)
    # V alone, then K and V
    for k in (fine, bad):
        q.kv_append(s.cache, k, bad, s.slots[at].contiguous())
        mask, _ = q.tree_mask(parents.to(dev))
        queries = _rows((3, nodes, rep, dim), dtype, 6, loud=False)
        got = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask))
        for b in range(3):
            see = seen_by(rows[b], 120, 0)
            ref, tol = bounded(queries, s, b, see)
            for i in range(nodes):
                if lost[b] is not None and lost[b] in path_up(rows[b], i):
                    assert not np.isfinite(got[b, i]).any(), (b, i)
                else:
                    within(got[b, i], ref[i], tol[i])
        assert (got[0, 9] == 0).all()


@pytest.mark.parametrize("nodes,rep,dim,group,dtype", FORMS)
def test_tokens_of_the_context_that_are_not_finite(nodes, rep, dim, group, dtype):
    """A token before the tree that the window leaves to some nodes only."""
    import bit_affine_quantized_qmv_amd as q
    window = 9
    s = Setup([150], 1, dim, group, 16, dtype, seed=15)
    dev = s.len_dev.device
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32)[None].clone()
    parents[0, nodes // 2:] = torch.arange(nodes // 2, nodes, dtype=torch.int32) - nodes // 2 - 1     # a second chain
    mask, depth = q.tree_mask(parents.to(dev), window=window)
    c = 150 - nodes
    bad = torch.full((1, 1, dim), float("inf"), dtype=TORCH_DTYPE[dtype], device=dev)
    q.kv_append(s.cache, bad, bad, s.slots[c - 5:c - 4].contiguous())
    queries = _rows((1, nodes, rep, dim), dtype, 6, loud=False)
    got = values(q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask, depth, window=window))[0]
    see = seen_by(parents[0].tolist(), 150, window)
    ref, tol = bounded(queries, s, 0, see)
    assert see[:, c - 5].any() and not see[:, c - 5].all()
    for i in range(nodes):
        if see[i, c - 5]:
            assert not np.isfinite(got[i]).any(), i
        else:
            within(got[i], ref[i], tol[i])
