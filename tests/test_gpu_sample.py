"""Sampling against a float64 reference of the definition, and exact cases."""
import math

import numpy as np
import pytest
import torch

from qmm_testlib import TORCH_DTYPE, require_gpu, values

pytestmark = pytest.mark.gpu

# Relative error of a weight: the float32 quotient (l - max) / T has two roundings, so z is off
# by |z| 2^-23 at most, and weights below e^-28 count for nothing; the exponential adds 2^-22.
REL = 2.0 ** -17


def floor24(x):
    return math.floor(min(max(float(x), 0.0), 1.0) * 2 ** 24) / 2 ** 24


def kept(l, t, k, p, min_p):
    """(columns in descending order, their float64 weights, cumulative weights) that a row keeps."""
    ok = np.flatnonzero(~np.isnan(l) & (l > -np.inf))
    order = ok[np.argsort(-l[ok], kind="stable")]
    if order.size == 0:
        return order, np.zeros(0)
    top = l[order[0]]
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / t) if t > 0 else 0.0)
    if t <= 0:
        order, w = order[:1], w[:1]
    if 0 < k < order.size:
        order, w = order[:k], w[:k]
    before = np.cumsum(w) - w
    keep = (before < floor24(p) * w.sum()) & (w >= min_p)
    keep[0] = True
    return order[keep], w[keep]


def check_row(index, prob, l, u, t, k, p, min_p):
    """The drawn column is one whose interval holds the target, up to the weights' errors; a
    column at the edge of the top-p or min-p cut may fall on either side of it."""
    loose = kept(l, t, k, min(1.0, p * (1 + 4 * REL) + 2.0 ** -23), min_p * (1 - 4 * REL))
    tight = kept(l, t, k, p * (1 - 4 * REL), min_p * (1 + 4 * REL))
    if loose[0].size == 0:
        assert index == -1 and prob == 0.0
        return
    assert index in loose[0], (index, loose[0][:5])
    ok = False
    for order, w in (loose, tight):
        by = np.argsort(order, kind="stable")
        cols, ww = order[by], w[by]
        cum = np.cumsum(ww)
        slack = 4 * REL * cum[-1]
        target = min(floor24(u), 1 - 2.0 ** -24) * cum[-1]
        at = np.flatnonzero(cols == index)
        if at.size and cum[at[0]] + slack > target and cum[at[0]] - ww[at[0]] - slack <= target:
            ok = ok or abs(prob - ww[at[0]] / cum[-1]) <= 8 * REL * ww[at[0]] / cum[-1] + 2.0 ** -39
    assert ok, (index, prob, u)


def logits_of(rows, n, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, n, generator=g)).to(TORCH_DTYPE[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,rows,pad", [(1, 3, 0), (2, 4, 1), (7, 5, 0), (511, 8, 1), (512, 3, 0), (513, 9, 3),
                                        (2049, 17, 0), (8192, 6, 8), (20011, 33, 5), (151936, 5, 0)])
def test_sample_matches_float64(n, rows, pad, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    big = logits_of(rows, n + pad, dtype, n + rows)
    x = big[:, pad // 2:pad // 2 + n]                       # odd row starts: 2-byte aligned rows
    rng = np.random.default_rng(n)
    for round_ in range(3):
        t = np.where(rng.random(rows) < 0.15, 0.0, rng.uniform(0.3, 1.7, rows)).astype(np.float32)
        k = np.where(rng.random(rows) < 0.5, 0, rng.integers(1, 2 * n + 2, rows)).astype(np.int32)
        if round_ == 1:
            k = np.minimum(k, 60)
        p = np.where(rng.random(rows) < 0.4, 1.0, rng.uniform(0.05, 0.999, rows)).astype(np.float32)
        m = np.where(rng.random(rows) < 0.6, 0.0, rng.uniform(0.0, 0.3, rows)).astype(np.float32)
        u = rng.random(rows).astype(np.float32)
        u[0] = 0.0
        u[-1] = 1.0
        dx = big.to(dev)[:, pad // 2:pad // 2 + n]
        idx, prob = q.sample(dx, torch.from_numpy(u).to(dev), torch.from_numpy(t).to(dev),
                             torch.from_numpy(k).to(dev), torch.from_numpy(p).to(dev), torch.from_numpy(m).to(dev))
        torch.cuda.synchronize()
        l = values(x)
        for r in range(rows):
            check_row(int(idx[r]), float(prob[r]), l[r], u[r], float(t[r]), int(k[r]), float(p[r]), float(m[r]))


def test_sample_equal_logits_are_exact():
    """Equal logits: the draw is floor(u * count) among the kept columns, lower columns first."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    n = 3000
    x = torch.full((64, n), 1.5, dtype=torch.float16)
    x[:, 100:200] = -math.inf                               # never drawn
    x[:, 300] = float("nan")
    open_cols = [c for c in range(n) if not 100 <= c < 200 and c != 300]
    u = torch.arange(64, dtype=torch.float32) / 64
    for k, p in ((0, 1.0), (1000, 1.0), (0, 0.5), (1000, 0.25), (7, 1.0), (0, 2.0 ** -12)):
        count = min(k, len(open_cols)) if k else len(open_cols)
        count = max(1, math.ceil(p * count))
        idx, prob = q.sample(x.to(dev), u.to(dev), temperature=0.7, top_k=k, top_p=p)
        torch.cuda.synchronize()
        for r in range(64):
            assert int(idx[r]) == open_cols[(r * count) // 64], (k, p, r)
            assert abs(float(prob[r]) - 1 / count) < 1e-9 + 1e-6 / count


def test_sample_rows_with_nothing_and_infinities():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    for dtype in ("bf16", "fp16"):
        lowest = torch.finfo(TORCH_DTYPE[dtype]).min
        x = torch.zeros(6, 1000, dtype=TORCH_DTYPE[dtype])
        x[0] = -math.inf
        x[1] = float("nan")
        x[2], x[2, [5, 900]] = -1.0, math.inf               # +inf takes everything
        x[3], x[3, 77] = float("nan"), -3.0
        x[4] = lowest                                       # a mask of the lowest value everywhere
        x[5], x[5, 400] = lowest, 0.25
        u = torch.tensor([0.5, 0.5, 0.75, 0.5, 0.5, 0.999], device=dev)
        want = [-1, -1, 900, 77, 500, 400]
        for kw in ({}, {"top_k": 1000}, {"top_p": 1.0 - 2.0 ** -24}, {"min_p": 1.0}):
            idx, prob = q.sample(x.to(dev), u, **kw)
            torch.cuda.synchronize()
            assert idx.tolist()[:4] == want[:4] and idx.tolist()[5] == want[5], (dtype, kw, idx)
            assert abs(idx.tolist()[4] - want[4]) <= 1
            assert prob.tolist()[:2] == [0.0, 0.0] and prob.tolist()[2] == 0.5 and prob.tolist()[3] == 1.0
        idx, _ = q.sample(x.to(dev), u, temperature=0.0)
        torch.cuda.synchronize()
        assert idx.tolist() == [-1, -1, 5, 77, 0, 400]


def test_sample_settings_that_leave_the_first_maximum():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    x = logits_of(4, 5000, "bf16", 3)
    x[:, 4000] = x.float().amax() + 1
    x[:, 4001] = x[:, 4000]
    u = torch.full((4,), 0.99, device=dev)
    nan = float("nan")
    for kw in ({"temperature": 0.0}, {"temperature": -1.0}, {"temperature": nan}, {"top_k": 1}, {"top_p": 0.0},
               {"top_p": -2.0}, {"top_p": nan}, {"min_p": 1.5}, {"min_p": nan}):
        idx, prob = q.sample(x.to(dev), u, **kw)
        torch.cuda.synchronize()
        assert idx.tolist() == [4000] * 4 and prob.tolist() == [1.0] * 4, kw


def test_sample_same_result_for_any_split_stream_and_graph():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    x = logits_of(40, 30011, "fp16", 4).to(dev)
    g = torch.Generator().manual_seed(5)
    u = torch.rand(40, generator=g).to(dev)
    kw = dict(temperature=0.9, top_k=300, top_p=0.9, min_p=0.01)
    want, wprob = q.sample(x, u, **kw)
    for r in range(0, 40, 7):                               # one row: more, smaller chunks
        i1, p1 = q.sample(x[r:r + 1], u[r:r + 1], **kw)
        torch.cuda.synchronize()
        assert int(i1) == int(want[r]) and float(p1) == float(wprob[r])
    ws = q.sample_workspace(40, dev)
    ws.fill_(-1)
    idx, prob = torch.empty_like(want), torch.empty_like(wprob)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.sample(x, u, out_index=idx, out_prob=prob, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(idx, want) and torch.equal(prob, wprob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.sample(x, u, out_index=idx, out_prob=prob, workspace=ws, **kw)
    for _ in range(4):
        idx.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want) and torch.equal(prob, wprob)
        q.sample(x[:3], u[:3], workspace=ws, **kw)          # eager work between replays
        torch.cuda.synchronize()


def test_sample_frequencies_follow_the_weights():
    """4096 evenly spaced uniform numbers over one row hit each column its share of times."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    l = logits_of(1, 40, "bf16", 6, spread=1.5)
    rows = 4096
    u = ((torch.arange(rows) + 0.5) / rows).to(dev)
    idx, _ = q.sample(l.to(dev).expand(rows, 40).contiguous(), u, temperature=1.3)
    torch.cuda.synchronize()
    w = np.exp(values(l)[0] / 1.3)
    expect = rows * w / w.sum()
    got = np.bincount(idx.cpu().numpy(), minlength=40)
    assert np.abs(got - expect).max() <= 1.01


def test_sample_no_rows():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    idx, prob = q.sample(torch.empty(0, 9, dtype=torch.bfloat16, device=dev), torch.empty(0, device=dev))
    assert idx.shape == (0,) and prob.shape == (0,)
