"""Attention of trees with masks and depths of the caller's own, under a window: a tree that was
pruned keeps the depths that its nodes had, so they may pass its number of nodes."""
import numpy as np
import pytest
import torch

from qmm_testlib import values
from test_gpu_kv_cache import Setup, _rows
from test_gpu_tree import _ints
from tree_forms import shares_unpacked_values
from tree_testlib import masked_reference

pytestmark = pytest.mark.gpu

DEPTHS = [
    # length, nodes, heads, rep, dim, group, page, window, dtype, what runs
    (300, 9, 2, 4, 128, 64, 16, 40, "bf16"),          # 16 rows a workgroup
    (700, 21, 1, 2, 64, 32, 48, 200, "fp16"),
    (400, 20, 1, 2, 256, 64, 16, 65, "bf16"),
    (500, 64, 1, 4, 128, 64, 64, 100, "bf16"),        # two tiles of 16 rows per wave
    (600, 130, 1, 2, 128, 128, 16, 300, "fp16"),
    (500, 90, 1, 3, 128, 32, 16, 100, "bf16"),        # 16 rows a wave, many of a workgroup
    (700, 256, 1, 4, 64, 64, 16, 150, "fp16"),
    (900, 130, 1, 8, 256, 128, 32, 333, "bf16"),
]


@pytest.mark.parametrize("length,nodes,heads,rep,dim,group,page,window,dtype", DEPTHS)
@pytest.mark.parametrize("kind", ["far", "mixed", "low", "extreme"])
def test_depths_of_the_callers_own(length, nodes, heads, rep, dim, group, page, window, dtype, kind):
    import bit_affine_quantized_qmv_amd as q
    s = Setup([length], heads, dim, group, page, dtype, seed=dim + nodes)
    dev = s.len_dev.device
    g = np.random.RandomState(nodes + window)
    depth = {"far": lambda: g.randint(nodes, nodes + window + 40, nodes), "mixed": lambda: g.randint(0, length, nodes),
             "low": lambda: g.randint(-300, 3, nodes),
             "extreme": lambda: np.where(g.rand(nodes) < 0.5, 2 ** 31 - 1, -2 ** 31)}[kind]()
    sees = np.tril(g.rand(nodes, nodes) < 0.4)
    sees[np.arange(nodes), np.arange(nodes)] = True
    sees[nodes // 2] = False                                            # a row that sees nothing
    bits = np.zeros((nodes, (nodes + 31) // 32), np.uint32)
    for j in range(nodes):
        bits[:, j // 32] |= sees[:, j].astype(np.uint32) << np.uint32(j % 32)
    mask = torch.from_numpy(bits.view(np.int32)).to(dev)[None].contiguous()
    queries = _rows((1, nodes, heads * rep, dim), dtype, 77, loud=False)
    c = length - nodes
    see = np.zeros((nodes, length), bool)
    see[:, c:] = sees
    for i in range(nodes):
        if sees[i].any():                                               # a depth below 0 counts as 0
            see[i, max(0, min(c, c + max(0, int(depth[i])) - window + 1)):c] = True
    ref, tol = masked_reference(queries[0], s.k[0], s.v[0], see, group, dtype, dim ** -0.5,
                                shares_unpacked_values(nodes * rep, dim, group))
    for most in (None, length):
        y = q.kv_attend_tree(queries.to(dev), s.cache, s.table, s.len_dev, mask, _ints([depth.tolist()], dev),
                             window=window, max_length=most)
        err = np.abs(values(y[0]) - ref)
        assert (err <= tol).all(), "worst %.3g of the bound" % (err / np.maximum(tol, 1e-30)).max()
        assert (values(y[0, nodes // 2]) == 0).all()
