"""Forks into tables with fewer blocks than rows need: every block without an entry is reported, those of
kept tokens too."""
import pytest

from fork_testlib import cut_inputs, fork_rule
from test_gpu_fork_cuts import fork

pytestmark = pytest.mark.gpu


def test_kept_blocks_that_do_not_fit_are_counted():
    # 48 tokens in pages 0, 1 and 2, which a table of 2 blocks takes over: page 2 is lost, and free afterwards
    refs, table = [1, 1, 1, 0, 0], [[0, 1, 2]]
    assert fork(refs, table, [48], [0], 16, None, 2) == ([[0, 1]], [1, 1, 0, 0, 0], [-1], [-1], 1)
    # 40 tokens and room for 70: block 2 is kept in part, 3 and 4 are new
    assert fork(refs, table, [40], [0], 16, [70], 1) == ([[0]], [1, 0, 0, 0, 0], [-1], [-1], 4)
    # two such rows; a table of no blocks
    assert fork(refs, table, [48], [0, 0], 16, [48, 20], 1) == ([[0], [0]], [2, 0, 0, 0, 0], [-1, -1], [-1, -1], 3)
    assert fork(refs, table, [48], [0, -1], 16, [33, 5], 0) == ([[], []], [0, 0, 0, 0, 0], [-1, -1], [-1, -1], 4)
    # a kept block that had no page before the call is not counted again
    assert fork([1, 0, 1, 0, 0], [[0, -1, 2]], [48], [0], 16, None, 3) == ([[0, -1, 2]], [1, 0, 1, 0, 0], [-1], [-1], 0)
    # many blocks too few: at most 16384 of a row count
    assert fork([0, 0], [[]] * 0, [], [-1, -1], 16, [2 ** 31 - 1, 33], 1)[4] == 16384 + 2


@pytest.mark.parametrize("pages,batch,blocks,page,rows,new,spread", [
    (200, 4, 6, 16, 12, 3, 30), (4000, 3, 6, 48, 300, 2, 60), (9000, 20, 300, 16, 70, 150, 200), (60, 4, 6, 16, 30, 4, 30)])
def test_narrow_tables(pages, batch, blocks, page, rows, new, spread):
    for seed in range(5):
        refs, table, lengths, parents, want = cut_inputs(seed, pages, batch, blocks, page, rows, spread)
        for w in (want, None):
            assert fork(refs, table, lengths, parents, page, w, new) == \
                fork_rule(refs, table, lengths, parents, page, w, new), seed
