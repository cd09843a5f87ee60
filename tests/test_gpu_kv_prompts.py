"""Cache attention with more query rows per cached head than the single-token form takes (its
workgroups share a step's unpacked tokens over many query rows), against the same float64
reference and bounds; and arguments at their limits, for both forms."""
import pytest
import torch

from qmm_testlib import require_gpu
from test_gpu_kv_cache import Setup, _rows

pytestmark = pytest.mark.gpu

PROMPTS = [
    # lengths, q_len, heads, rep, dim, group, page, window, dtype
    ([540, 700], 540, 1, 1, 64, 64, 16, 0, "bf16"),
    ([300, 0, 7], 260, 1, 2, 64, 32, 32, 0, "fp16"),                # more queries than tokens: padded rows
    ([400, 70], 140, 2, 4, 128, 64, 64, 0, "bf16"),
    ([600], 260, 1, 2, 128, 128, 16, 100, "bf16"),
    ([530], 175, 1, 3, 128, 32, 48, 0, "fp16"),
    ([560, 520], 520, 1, 1, 256, 64, 16, 0, "bf16"),
    ([560], 513, 1, 1, 256, 32, 16, 50, "fp16"),
    ([200], 130, 1, 4, 256, 128, 16, 0, "bf16"),
    ([540, 90], 520, 1, 2, 64, 64, 16, 0, "bf16"),                  # as above with twice the rows and more
    ([300, 0, 7], 260, 1, 4, 64, 32, 32, 77, "fp16"),
    ([330], 300, 2, 4, 256, 64, 16, 0, "bf16"),
    ([560], 513, 1, 2, 256, 32, 16, 50, "fp16"),
    ([200], 260, 1, 4, 256, 128, 16, 0, "bf16"),
]


@pytest.mark.parametrize("lengths,q_len,heads,rep,dim,group,page,window,dtype", PROMPTS)
def test_prompt_matches_float64(lengths, q_len, heads, rep, dim, group, page, window, dtype):
    import bit_affine_quantized_qmv_amd as q
    s = Setup(lengths, heads, dim, group, page, dtype, seed=dim + q_len)
    dev = s.len_dev.device
    queries = _rows((len(lengths), q_len, heads * rep, dim), dtype, 78, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
    torch.cuda.synchronize()
    s.check(y, queries, dim ** -0.5, window=window)


@pytest.mark.parametrize("q_len", [270, 520])
def test_prompt_all_tokens_scale_and_strides(q_len):
    """causal=False, a negative scale, queries as a strided slice of a larger tensor."""
    import bit_affine_quantized_qmv_amd as q
    lengths, heads, rep, dim = [60, 1, 0, 200], 2, 2, 128
    s = Setup(lengths, heads, dim, 64, 16, "bf16", seed=5)
    dev = s.len_dev.device
    big = _rows((heads * rep + 2, len(lengths), q_len, dim + 8), "bf16", 6, loud=False)
    view = big.to(dev)[1:-1, :, :, :dim].permute(1, 2, 0, 3)
    y = q.kv_attend(view, s.cache, s.table, s.len_dev, scale=-0.21, causal=False)
    torch.cuda.synchronize()
    s.check(y, view.cpu(), -0.21, causal=False)


@pytest.mark.parametrize("q_len", [140, 260])
def test_prompt_masked_tokens_may_hold_anything(q_len):
    """NaN and infinite rows that a query does not see leave its output alone."""
    import bit_affine_quantized_qmv_amd as q
    n, window = 400, 64
    s = Setup([n], 1, 64, 32, 16, "bf16", seed=13)
    dev = s.len_dev.device
    queries = _rows((1, q_len, 4, 64), "bf16", 14, loud=False)
    clean = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
    bad = s.cache.data.clone()
    sb = 16 * 64 // 8
    side = sb + 2 * 16
    for token, word in ((n - 1, 0x7FFF7FFF), (0, 0x7F807F80), (n - q_len - window, 0x7FFF7FFF)):
        page = int(s.table[0, token // 16])
        for start in (0, side):
            for g in (0, 1):
                bad[page, 0, start + sb + g * 16 + token % 16] = word
    y = q.kv_attend(queries.to(dev), q.KVCache(bad, 16, 64, 32, torch.bfloat16), s.table, s.len_dev, window=window)
    torch.cuda.synchronize()
    assert torch.equal(y[0, :-1], clean[0, :-1])                # the last query alone sees token n - 1
    assert torch.isnan(y[0, -1].float()).all()


@pytest.mark.parametrize("q_len", [300, 520])
def test_prompt_a_missing_page_reaches_the_output_through_the_splits(q_len):
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


@pytest.mark.parametrize("q_len", [2, 600, 1100])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40])
def test_a_window_beyond_any_length_is_no_window(q_len, window):
    """Also where queries stand before the sequence (more queries than tokens)."""
    import bit_affine_quantized_qmv_amd as q
    s = Setup([40, 1], 1, 64, 32, 16, "bf16", seed=23)
    dev = s.len_dev.device
    queries = _rows((2, q_len, 1, 64), "bf16", 24, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
    torch.cuda.synchronize()
    s.check(y, queries, 64 ** -0.5)


@pytest.mark.parametrize("q_len", [3, 520, 1050])
def test_scale_zero_is_the_mean_of_what_a_query_sees(q_len):
    import bit_affine_quantized_qmv_amd as q
    s = Setup([77, 2, 0], 1, 64, 32, 16, "fp16", seed=25)
    dev = s.len_dev.device
    queries = _rows((3, q_len, 1, 64), "fp16", 26, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, scale=0.0)
    torch.cuda.synchronize()
    s.check(y, queries, 0.0)


def test_tensors_of_one_call_are_on_one_gpu():
    import bit_affine_quantized_qmv_amd as q
    s = Setup([20], 1, 64, 32, 16, "bf16", seed=27)
    queries = _rows((1, 1, 2, 64), "bf16", 28)
    rows = _rows((20, 1, 64), "bf16", 29)
    with pytest.raises(ValueError, match="one GPU"):
        q.kv_append(s.cache, rows, rows, s.slots)
    with pytest.raises(ValueError, match="one GPU"):
        q.kv_attend(queries, s.cache, s.table, s.len_dev)
    with pytest.raises(ValueError, match="one GPU"):
        q.sample(torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, device=s.len_dev.device))


def test_a_pool_past_32_bit_offsets():
    """The same rows at the start of a small pool and at the end of one of 9 GB (more than 2^31
    words): the same bits come back, and the same outputs."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    page, heads, dim, group, n, last = 64, 8, 128, 32, 300, 110000
    if torch.cuda.mem_get_info(dev)[0] < 16 << 30:
        pytest.skip("needs 16 GB of free GPU memory")
    small = q.kv_cache(8, page, heads, dim, group, "bf16", dev)
    large = q.kv_cache(last, page, heads, dim, group, "bf16", dev)
    assert large.data.numel() > 2 ** 31
    blocks = -(-n // page)
    k, v = (_rows((n, heads, dim), "bf16", seed).to(dev) for seed in (31, 32))
    near = torch.arange(blocks, dtype=torch.int32, device=dev)[None]
    far = last - 1 - near
    results = []
    for cache, table in ((small, near), (large, far)):
        j = torch.arange(n, device=dev)
        slots = (table[0, j // page] * page + j % page).int()
        q.kv_append(cache, k, v, slots)
        lengths = torch.tensor([n], dtype=torch.int32, device=dev)
        outs = [q.kv_attend(_rows((1, q_len, 2 * heads, dim), "bf16", 33).to(dev), cache, table, lengths)
                for q_len in (1, 150)]
        results.append([*q.kv_read(cache, slots), *outs])
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert not torch.isnan(a.float()).any() and torch.equal(a, b)
