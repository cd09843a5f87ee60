"""The 4-bit key/value cache against float64 references: append and read bit for bit,
attention within the bound of its stated roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_testlib import attend_reference
from qmm_testlib import TORCH_DTYPE, half_bits, require_gpu, values

pytestmark = pytest.mark.gpu


def _rows(shape, dtype, seed, loud=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if loud:
        x = x * (1 + 6 * (torch.rand(*shape[1:], generator=g) < 0.05))
    return x.to(TORCH_DTYPE[dtype])


def _poison(cache):
    """NaN scales and biases everywhere (the pattern is NaN in both types)."""
    cache.data.fill_(0x7FFF7FFF)


def _expected_rows(x, group, dtype):
    flat = x.reshape(-1, x.shape[-1])
    q = O.quantize(flat.float().numpy(), group, 4, dtype)
    bits = O.dequantize_dtype(q["codes"], q["scales_bits"], q["biases_bits"], group, dtype)
    return bits.reshape(tuple(x.shape))


@pytest.mark.parametrize("dim,group,page,heads,dtype", [
    (64, 32, 16, 3, "bf16"), (64, 64, 48, 1, "fp16"), (128, 32, 64, 2, "fp16"), (128, 64, 16, 5, "bf16"),
    (128, 128, 256, 2, "bf16"), (256, 32, 32, 2, "bf16"), (256, 64, 16, 1, "fp16"), (256, 128, 80, 3, "fp16")])
def test_append_then_read_is_the_codec(dim, group, page, heads, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    pages, tokens = 5, 41
    cache = q.kv_cache(pages, page, heads, dim, group, dtype, dev)
    _poison(cache)
    before = cache.data.clone()
    k, v = _rows((tokens, heads, dim), dtype, dim + group), _rows((tokens, heads, dim), dtype, dim + group + 1)
    k[3, 0] = 0.25                      # a constant row: s = 0
    v[5] = 0.0
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(page))[:tokens].to(torch.int32)
    # strided inputs, as slices of one projection's output
    both = torch.zeros(tokens, heads + 1, 2, dim, dtype=k.dtype)
    both[:, :heads, 0], both[:, :heads, 1] = k, v
    both = both.to(dev)
    q.kv_append(cache, both[:, :heads, 0], both[:, :heads, 1], slots.to(dev))
    gk, gv = q.kv_read(cache, slots.to(dev))
    torch.cuda.synchronize()
    assert np.array_equal(half_bits(gk), _expected_rows(k, group, dtype))
    assert np.array_equal(half_bits(gv), _expected_rows(v, group, dtype))
    # every other slot still holds what was there: clear the written ones in both and compare
    for c in (cache.data, before):
        tmp = q.KVCache(c, page, dim, group, k.dtype)
        zero = torch.zeros(tokens, heads, dim, dtype=k.dtype, device=dev)
        q.kv_append(tmp, zero, zero, slots.to(dev))
    torch.cuda.synchronize()
    assert torch.equal(cache.data, before)


def test_append_skips_and_read_poisons_slots_outside():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    cache = q.kv_cache(2, 16, 2, 64, 32, "bf16", dev)
    k = _rows((4, 2, 64), "bf16", 3).to(dev)
    slots = torch.tensor([-1, 31, 32, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    q.kv_append(cache, k, k, slots)
    other = q.kv_cache(2, 16, 2, 64, 32, "bf16", dev)
    q.kv_append(other, k[1:2], k[1:2], slots[1:2])
    gk, gv = q.kv_read(cache, slots)
    torch.cuda.synchronize()
    assert torch.equal(cache.data, other.data)
    assert np.isnan(values(gk[[0, 2, 3]])).all() and np.isnan(values(gv[[0, 2, 3]])).all()
    assert np.array_equal(half_bits(gk[1]), _expected_rows(k[1].cpu(), 32, "bf16"))
    q.kv_append(cache, k[:0], k[:0], slots[:0])
    assert q.kv_read(cache, slots[:0])[0].shape == (0, 2, 64)


class Setup:
    """Sequences of the given lengths in a shuffled page pool whose every other slot is NaN."""

    def __init__(self, lengths, heads, dim, group, page, dtype, seed=0):
        import bit_affine_quantized_qmv_amd as q
        dev = require_gpu()
        self.lengths, self.dim, self.group, self.dtype = lengths, dim, group, dtype
        blocks = [-(-n // page) for n in lengths]
        pages = sum(blocks) + 2
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
        width = max(max(blocks), 1) + 1
        table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        self.k, self.v, slots = [], [], []
        for i, (n, m) in enumerate(zip(lengths, blocks)):
            mine = [perm.pop() for _ in range(m)]
            table[i, :m] = torch.tensor(mine, dtype=torch.int32)
            slots += [mine[j // page] * page + j % page for j in range(n)]
            self.k.append(_rows((n, heads, dim), dtype, seed + 10 * i + 2))
            self.v.append(_rows((n, heads, dim), dtype, seed + 10 * i + 3))
        self.cache = q.kv_cache(pages, page, heads, dim, group, dtype, dev)
        _poison(self.cache)
        self.table = table.to(dev)
        self.len_dev = torch.tensor(lengths, dtype=torch.int32, device=dev)
        self.slots = torch.tensor(slots, dtype=torch.int32, device=dev)
        if slots:
            q.kv_append(self.cache, torch.cat(self.k).to(dev), torch.cat(self.v).to(dev), self.slots)

    def check(self, y, queries, scale, causal=True, window=0, skip=()):
        y = values(y)
        assert not np.isnan(np.delete(y, list(skip), axis=0)).any()
        for i, n in enumerate(self.lengths):
            if i in skip:
                continue
            ref, tol = attend_reference(queries[i], self.k[i], self.v[i], n, self.group, self.dtype, scale, causal,
                                        window)
            err = np.abs(y[i] - ref)
            assert (err <= tol).all(), "sequence %d (%d tokens): worst %.3g of the bound at %s" % (
                i, n, (err / np.maximum(tol, 1e-30)).max(), np.unravel_index((err - tol).argmax(), err.shape))


ATTEND = [
    # lengths, q_len, heads, rep, dim, group, page, window, dtype
    ([0, 1, 2, 31, 32, 33, 127, 128, 129, 300], 1, 2, 4, 128, 64, 16, 0, "bf16"),
    ([509], 1, 8, 4, 128, 64, 64, 0, "bf16"),
    ([1, 47, 48, 49, 700], 1, 1, 1, 64, 32, 48, 0, "fp16"),
    ([5, 260], 1, 3, 5, 64, 64, 32, 0, "bf16"),
    ([2500, 3], 1, 1, 8, 128, 128, 256, 0, "fp16"),
    ([130, 1025], 1, 2, 3, 128, 32, 16, 0, "bf16"),
    ([77, 400], 1, 2, 2, 256, 64, 16, 0, "bf16"),
    ([77, 200], 2, 1, 4, 256, 32, 32, 0, "fp16"),
    ([90, 333], 1, 1, 16, 256, 128, 64, 0, "bf16"),
    ([0, 1, 3, 40, 200], 5, 2, 4, 64, 32, 16, 0, "bf16"),           # more queries than tokens: padded rows
    ([500, 64, 20], 5, 1, 4, 64, 32, 16, 37, "fp16"),               # a window that starts inside a tile
    ([1000, 999], 3, 2, 2, 128, 64, 16, 1, "bf16"),                 # a window of the query's own token
    ([300], 17, 2, 2, 128, 64, 16, 0, "bf16"),                      # two row tiles
    ([150, 20], 50, 1, 2, 64, 64, 16, 0, "fp16"),
    ([400, 70], 70, 2, 4, 128, 64, 64, 0, "bf16"),                  # prompts: waves of their own rows
    ([330], 211, 1, 3, 128, 32, 48, 0, "fp16"),
    ([600], 130, 1, 2, 128, 128, 16, 100, "bf16"),
    ([260], 260, 1, 1, 64, 64, 16, 0, "bf16"),
    ([300, 0], 150, 1, 1, 64, 32, 32, 0, "fp16"),
    ([200], 140, 1, 1, 256, 64, 16, 0, "bf16"),
    ([210], 129, 1, 1, 256, 32, 16, 50, "fp16"),
]


@pytest.mark.parametrize("lengths,q_len,heads,rep,dim,group,page,window,dtype", ATTEND)
def test_attend_matches_float64(lengths, q_len, heads, rep, dim, group, page, window, dtype):
    import bit_affine_quantized_qmv_amd as q
    s = Setup(lengths, heads, dim, group, page, dtype, seed=dim + q_len)
    dev = s.len_dev.device
    queries = _rows((len(lengths), q_len, heads * rep, dim), dtype, 77, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
    again = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window,
                        max_length=max(lengths) or 1)
    torch.cuda.synchronize()
    s.check(y, queries, dim ** -0.5, window=window)
    s.check(again, queries, dim ** -0.5, window=window)


@pytest.mark.parametrize("q_len,rep,dtype", [(1, 4, "bf16"), (7, 2, "fp16"), (80, 2, "bf16")])
def test_attend_all_tokens_scale_and_strides(q_len, rep, dtype):
    """causal=False, a given scale, queries as a strided slice of a larger tensor."""
    import bit_affine_quantized_qmv_amd as q
    lengths, heads, dim = [60, 1, 0, 200], 2, 128
    s = Setup(lengths, heads, dim, 64, 16, dtype, seed=5)
    dev = s.len_dev.device
    big = _rows((heads * rep + 2, len(lengths), q_len, dim + 8), dtype, 6, loud=False)
    view = big.to(dev)[1:-1, :, :, :dim].permute(1, 2, 0, 3)
    y = q.kv_attend(view, s.cache, s.table, s.len_dev, scale=0.21, causal=False)
    torch.cuda.synchronize()
    s.check(y, view.cpu(), 0.21, causal=False)


def test_attend_sharp_scores():
    """Scores far apart (the running maximum rises late and by much) and a negative scale."""
    import bit_affine_quantized_qmv_amd as q
    for dtype in ("bf16", "fp16"):
        s = Setup([333], 1, 128, 64, 16, dtype, seed=9)
        dev = s.len_dev.device
        queries = 8 * _rows((1, 1, 4, 128), dtype, 10, loud=False)
        for scale in (1.0, -0.5):
            y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, scale=scale)
            torch.cuda.synchronize()
            s.check(y, queries, scale)


def test_attend_largest_fp16_values():
    """Values over fp16's whole range: unnormalised probabilities times V's scales stay finite."""
    import bit_affine_quantized_qmv_amd as q
    s = Setup([64], 1, 64, 64, 16, "fp16", seed=11)
    dev = s.len_dev.device
    v = torch.where(torch.rand(64, 1, 64, generator=torch.Generator().manual_seed(1)) < 0.5, 65504.0, -65504.0).half()
    s.v[0] = v
    q.kv_append(s.cache, s.k[0].to(dev), v.to(dev), s.slots)
    queries = _rows((1, 1, 2, 64), "fp16", 12, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev)
    torch.cuda.synchronize()
    s.check(y, queries, 64 ** -0.5)


def test_attend_masked_tokens_may_hold_anything():
    """NaN and infinite rows that a query does not see leave its output alone: later tokens
    under the causal mask, earlier ones outside the window."""
    import bit_affine_quantized_qmv_amd as q
    for q_len in (4, 40):
        s = Setup([200], 1, 64, 32, 16, "bf16", seed=13)
        dev = s.len_dev.device
        queries = _rows((1, q_len, 4, 64), "bf16", 14, loud=False)
        window = 64
        clean = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
        bad = s.cache.data.clone()
        sb = 16 * 64 // 8                                       # the (s, b) words of a page's side
        side = sb + 2 * 16
        for token, word in ((199, 0x7FFF7FFF), (0, 0x7F807F80), (200 - q_len - window, 0x7FFF7FFF)):
            page = int(s.table[0, token // 16])
            for start in (0, side):
                for g in (0, 1):
                    bad[page, 0, start + sb + g * 16 + token % 16] = word
        y = q.kv_attend(queries.to(dev), q.KVCache(bad, 16, 64, 32, torch.bfloat16), s.table, s.len_dev,
                        window=window)
        torch.cuda.synchronize()
        assert torch.equal(y[0, :-1], clean[0, :-1])            # the last query alone sees token 199
        assert torch.isnan(y[0, -1].float()).all()


def test_attend_bad_lengths_and_pages_give_nan():
    import bit_affine_quantized_qmv_amd as q
    s = Setup([100, 100, 100, 100], 1, 64, 32, 16, "bf16", seed=15)
    dev = s.len_dev.device
    queries = _rows((4, 1, 2, 64), "bf16", 16, loud=False)
    table = s.table.clone()
    table[1, 3] = -1                       # a page that is needed
    table[3, 7:] = 10 ** 6                 # entries past the sequence are never read
    lengths = torch.tensor([100, 100, 129, 100], dtype=torch.int32, device=dev)
    for workers in (1, 2):                 # whole, and split over workgroups
        y = q.kv_attend(queries.to(dev), s.cache, table, lengths, max_length=128 if workers == 1 else None)
        if workers == 2:
            lengths = torch.tensor([100, 100, -1, 100], dtype=torch.int32, device=dev)
            y = q.kv_attend(queries.to(dev), s.cache, table, lengths)
        torch.cuda.synchronize()
        assert torch.isnan(y[1].float()).all() and torch.isnan(y[2].float()).all()
        s.check(y, queries, 64 ** -0.5, skip=(1, 2))


@pytest.mark.parametrize("q_len", [1, 140])
def test_attend_a_missing_page_reaches_the_output_through_the_splits(q_len):
    """One page of a long sequence is not in the pool: the queries that need it are NaN, the
    ones before it (and other sequences) are not."""
    import bit_affine_quantized_qmv_amd as q
    s = Setup([3000, 2900], 1, 64, 32, 16, "bf16", seed=21)
    dev = s.len_dev.device
    queries = _rows((2, q_len, 2, 64), "bf16", 22, loud=False)
    for block in (1000 // 16, (3000 - q_len // 2 - 1) // 16):
        table = s.table.clone()
        table[0, block] = 10 ** 6
        y = q.kv_attend(queries.to(dev), s.cache, table, s.len_dev)
        torch.cuda.synchronize()
        nan = torch.isnan(y.float())
        needs = torch.tensor([3000 - q_len + i >= 16 * block for i in range(q_len)])
        assert nan[0][needs].all() and not nan[0][~needs].any() and not nan[1].any()


def test_attend_same_bits_again_on_another_stream_and_in_a_graph():
    import bit_affine_quantized_qmv_amd as q
    s = Setup([900, 17, 300], 2, 128, 64, 16, "bf16", seed=17)
    dev = s.len_dev.device
    queries = _rows((3, 1, 8, 128), "bf16", 18, loud=False).to(dev)
    want = q.kv_attend(queries, s.cache, s.table, s.len_dev)
    ws = q.kv_attend_workspace(queries, s.cache, 1024)
    ws.fill_(float("nan"))
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.kv_attend(queries, s.cache, s.table, s.len_dev, out=out, max_length=912, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    same_plan = q.kv_attend(queries, s.cache, s.table, s.len_dev, max_length=912)
    torch.cuda.synchronize()
    assert torch.equal(out, same_plan)
    pad = torch.full((3,), -1, dtype=torch.int32, device=dev)    # slots that append nothing
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.kv_append(s.cache, queries[:, 0, :2], queries[:, 0, 2:4], pad)
        q.kv_attend(queries, s.cache, s.table, s.len_dev, out=out, max_length=912, workspace=ws)
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, same_plan)
        q.kv_attend(queries[:1], s.cache, s.table[:1], s.len_dev[:1])     # eager work between replays
        torch.cuda.synchronize()


def test_attend_no_queries_is_a_no_op():
    import bit_affine_quantized_qmv_amd as q
    s = Setup([10], 1, 64, 32, 16, "bf16")
    e = torch.empty(1, 0, 2, 64, dtype=torch.bfloat16, device=s.len_dev.device)
    assert q.kv_attend(e, s.cache, s.table, s.len_dev).shape == (1, 0, 2, 64)
    assert q.kv_attend(e.view(0, 1, 2, 64), s.cache, s.table[:0], s.len_dev[:0]).shape == (0, 1, 2, 64)
