"""Reference of forks of block tables, entry by entry from the definition (plain Python on the CPU).
A row writes from its kept tokens on, so no page from there on may be another row's: the first row
of a parent keeps its old pages from the block on that no other row of the parent shares."""
from __future__ import annotations

import numpy as np


def kept_tokens(lengths, parents, want):
    """(length, want, kept) of every row."""
    rows = []
    for i, p in enumerate(parents):
        length = max(0, lengths[p]) if 0 <= p < len(lengths) else 0
        w = length if want is None else max(0, want[i])
        rows.append((length, w, min(length, w)))
    return rows


def fork_rule(refs, table, lengths, parents, page, want, blocks):
    """(new table, refs, copy_src, copy_dst, short) as lists."""
    pages = len(refs)
    sizes = kept_tokens(lengths, parents, want)
    free = [p for p in range(pages) if refs[p] == 0]
    out, src, dst, short = [], [], [], 0
    for i, p in enumerate(parents):
        has = 0 <= p < len(table)
        _, w, keep = sizes[i]
        others = [o for o, x in enumerate(parents) if x == p and o != i]
        shared = max([sizes[o][2] // page for o in others], default=0)     # blocks that another row names
        first = has and all(o > i for o in others)
        row, copy = [-1] * blocks, (-1, -1)
        for j in range(min(blocks, -(-w // page))):
            was = table[p][j] if has and j < len(table[p]) and 0 <= table[p][j] < pages else -1
            if j < keep // page or (first and was >= 0 and refs[was] == 1 and j >= shared):
                row[j] = was
                continue
            row[j] = free.pop(0) if free else -1
            short += row[j] < 0
            if j == keep // page and keep % page and was >= 0 and row[j] >= 0:
                copy = (was, row[j])
        short += min(16384, max(0, -(-w // page) - blocks))
        out.append(row)
        src.append(copy[0])
        dst.append(copy[1])
    new = list(refs)
    for rows, step in ((table, -1), (out, 1)):
        for row in rows:
            for p in row:
                if 0 <= p < pages:
                    new[p] += step
    return out, new, src, dst, short


def shared_writes(table, refs, lengths, parents, page, want):
    """Entries (row, block) of a new table that their row writes and another row names too."""
    sizes = kept_tokens(lengths, parents, want)
    return [(i, j) for i, row in enumerate(table) for j, p in enumerate(row)
            if p >= 0 and j >= sizes[i][2] // page and refs[p] != 1]


def cut_inputs(seed, pages, batch, blocks, page, rows, spread, from_start=True):
    """(refs, table, lengths, parents, want): sequences with pages of their own, rows that keep any
    part of them, many of one parent."""
    g = np.random.RandomState(seed)
    free = g.permutation(pages).tolist()
    lengths = g.randint(1, blocks * page + 1, batch).tolist()
    table = [[free.pop() for _ in range(-(-n // page))] for n in lengths]
    table = [row + [-1] * (blocks - len(row)) for row in table]
    refs = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    parents = g.randint(0, batch, rows).tolist()
    low = (lambda n: 0) if from_start else (lambda n: max(0, n - spread))
    want = [int(g.randint(low(lengths[p]), lengths[p] + spread)) for p in parents]
    return refs, table, lengths, parents, want
