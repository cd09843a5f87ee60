"""References of the tests of drafted trees, moves, forks and grouped products, from the
definitions (numpy and plain Python on the CPU)."""
from __future__ import annotations

import numpy as np
import torch

from kv_precise import F32, PROMPT, SINGLE
from kv_testlib import cached_parts, half_ulp
from qmm_testlib import values


def path_up(parents, i):
    """Node i and its ancestors, nearest first; [] where one of them is no node."""
    path = []
    while i != -1:
        if i < 0 or not -1 <= parents[i] < i:
            return []
        path.append(i)
        i = parents[i]
    return path


def random_parents(batch, nodes, seed, drop=0.0):
    """Random trees int32 [batch, nodes]: node 0 a root, now and then another; some are no nodes."""
    g = np.random.RandomState(seed)
    p = np.full((batch, nodes), -1, np.int64)
    for i in range(1, nodes):
        p[:, i] = np.minimum((i * g.rand(batch) ** 0.5).astype(np.int64), i - 1)
    p[g.rand(batch, nodes) < 0.04] = -1
    no = g.rand(batch, nodes) < drop
    p[no] = np.where(g.rand(no.sum()) < 0.5, -2, nodes + 5)
    return torch.from_numpy(p.astype(np.int32))


def seen_by(parents, length, window):
    """bool [nodes, length]: what each node of a tree that ends a sequence sees."""
    n = len(parents)
    see = np.zeros((n, length), bool)
    c = length - n
    for i in range(n):
        path = path_up(parents, i)
        if path:
            see[i, max(0, c + len(path) - window) if window else 0:c] = True
            see[i, [c + u for u in (path[:window] if window else path)]] = True
    return see


def masked_reference(q, k, v, see, group, dtype, scale, prompt):
    """One sequence: q [n, q_heads, d], k and v [length, heads, d] as appended, see bool
    [n, length].  (out, tol) float64 with the bounds of the stated operands (kv_precise)."""
    n, q_heads, d = q.shape
    rep = q_heads // k.shape[1]
    qv = values(q)
    out, tol = np.zeros((n, q_heads, d)), np.zeros((n, q_heads, d))
    ks, kc, kb = cached_parts(k, group, dtype)
    vs, vc, vb = cached_parts(v, group, dtype)
    kk, vv, codes = ks * kc + kb, vs * vc + vb, vs * vc
    k_size, v_size = ks * kc + np.abs(kb), codes + np.abs(vb)
    for i in range(n):
        at = np.flatnonzero(see[i])
        if not len(at):
            continue
        for h in range(q_heads):
            g = h // rep
            s = scale * (kk[at, g] @ qv[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv[at, g]
            e = w * (F32 * (1 + abs(scale) * (k_size[at, g] @ np.abs(qv[i, h]))))
            operands = PROMPT[dtype] * (w @ np.abs(vv[at, g])) if prompt else SINGLE * (w @ codes[at, g])
            tol[i, h] = operands + e @ v_size[at, g] + np.abs(out[i, h]) * e.sum()
    return out, tol + half_ulp(np.abs(out) + tol, dtype)


def accept_reference(parents, tokens, sampled):
    """(path, last) of one tree."""
    if parents[0] != -1:
        return [], -1
    path = [0]
    while True:
        l = path[-1]
        fits = [i for i in range(l + 1, len(parents)) if parents[i] == l and tokens[i] == sampled[l]]
        if not fits:
            return path, sampled[l]
        path.append(fits[0])


def fork_reference(refs, table, lengths, parents, page, want, blocks):
    """(new table, refs, copy_src, copy_dst, short) as lists, entry by entry."""
    pages = len(refs)
    old = lambda p, j: table[p][j] if 0 <= p < len(table) and j < len(table[p]) and 0 <= table[p][j] < pages else -1  # noqa: E731
    free = [p for p in range(pages) if refs[p] == 0]
    out, src, dst, short, seen = [], [], [], 0, set()
    for i, p in enumerate(parents):
        has = 0 <= p < len(table)
        length = max(0, lengths[p]) if has else 0
        w = length if want is None else max(0, want[i])
        keep = min(length, w)
        row, copy = [-1] * blocks, (-1, -1)
        for j in range(blocks):
            page_was = old(p, j) if has else -1
            if j < keep // page:
                row[j] = page_was
            elif j < -(-w // page):
                if has and p not in seen and page_was >= 0 and refs[page_was] == 1:
                    row[j] = page_was
                else:
                    row[j] = free.pop(0) if free else -1
                    short += row[j] < 0
                    if j == keep // page and keep % page and page_was >= 0 and row[j] >= 0:
                        copy = (page_was, row[j])
        short += min(16384, max(0, -(-w // page) - max(blocks, keep // page)))
        if has:
            seen.add(p)
        out.append(row)
        src.append(copy[0])
        dst.append(copy[1])
    new = list(refs)
    for row in table:
        for p in row:
            if 0 <= p < pages:
                new[p] -= 1
    for row in out:
        for p in row:
            if p >= 0:
                new[p] += 1
    return out, new, src, dst, short
