"""CPU tests of the forks' reference: no row writes a page that another one names, whatever the rows
keep."""
import pytest

from fork_testlib import cut_inputs, fork_rule, shared_writes
from tree_testlib import fork_reference

PARENT = ([1, 1, 1, 1, 0, 0, 0, 0], [[0, 1, 2, 3]], [56])      # 56 tokens in pages 0 to 3 of 16


def test_rows_cut_back_next_to_rows_that_keep_more():
    # the first row stays in block 1, of which the second one keeps every token: a page of its own
    assert fork_rule(*PARENT, [0, 0], 16, [20, 56], 4) == \
        ([[0, 4, -1, -1], [0, 1, 2, 5]], [2, 1, 1, 0, 1, 1, 0, 0], [1, 3], [4, 5], 0)
    # a row that keeps more comes first: only it stays in its last page
    assert fork_rule(*PARENT, [0, 0], 16, [56, 20], 4) == \
        ([[0, 1, 2, 3], [0, 4, -1, -1]], [2, 1, 1, 1, 1, 0, 0, 0], [-1, 1], [-1, 4], 0)
    # rows that end in the same block: the first has it
    assert fork_rule(*PARENT, [0, 0], 16, [20, 30], 4) == \
        ([[0, 1, -1, -1], [0, 4, -1, -1]], [2, 1, 0, 0, 1, 0, 0, 0], [-1, 1], [-1, 4], 0)


@pytest.mark.parametrize("seed", range(30))
def test_no_row_writes_what_another_names(seed):
    refs, table, lengths, parents, want = cut_inputs(seed, 200, 4, 6, 16, 12, 30)
    out, after, _, _, short = fork_rule(refs, table, lengths, parents, 16, want, 8)
    assert short == 0 and not shared_writes(out, after, lengths, parents, 16, want)


@pytest.mark.parametrize("seed", range(10))
def test_rows_that_keep_everything_are_those_of_equal_rows(seed):
    """Without cuts the first row's claim does not depend on the others."""
    refs, table, lengths, parents, want = cut_inputs(seed, 200, 4, 6, 16, 12, 30)
    want = [max(w, lengths[p]) for w, p in zip(want, parents)]
    assert fork_rule(refs, table, lengths, parents, 16, want, 8) == \
        fork_reference(refs, table, lengths, parents, 16, want, 8)
