"""Prompt attention where all of a row's scores are far from zero: softmax does not depend on a
common offset, so the outputs have to be as right as near zero (and finite)."""
import pytest
import torch

from test_gpu_kv_cache import Setup, _rows

pytestmark = pytest.mark.gpu

FORMS = [
    # lengths, q_len, heads, rep, dim, group, window, dtype: 256 rows or more at 128, 1024 at 64 and 256
    ([300, 131], 130, 1, 2, 128, 64, 0, "bf16"),
    ([300], 130, 1, 2, 128, 128, 40, "fp16"),
    ([600, 520], 520, 1, 2, 64, 32, 0, "fp16"),
    ([600], 520, 1, 2, 64, 64, 100, "bf16"),
    ([530], 513, 1, 2, 256, 128, 0, "bf16"),
]


@pytest.mark.parametrize("offset", [-5000.0, -200.0, -95.0, 200.0])
@pytest.mark.parametrize("lengths,q_len,heads,rep,dim,group,window,dtype", FORMS)
def test_prompt_scores_with_a_common_offset(lengths, q_len, heads, rep, dim, group, window, dtype, offset):
    """One channel of every key holds 24 and of every query offset * dim^0.5 / 24."""
    import bit_affine_quantized_qmv_amd as q
    s = Setup(lengths, heads, dim, group, 16, dtype, seed=dim + q_len)
    dev = s.len_dev.device
    for k in s.k:
        k[:, :, 5] = 24.0
    q.kv_append(s.cache, torch.cat(s.k).to(dev), torch.cat(s.v).to(dev), s.slots)
    queries = _rows((len(lengths), q_len, heads * rep, dim), dtype, 78, loud=False)
    queries[..., 5] = offset * dim ** 0.5 / 24.0
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, window=window)
    torch.cuda.synchronize()
    s.check(y, queries, dim ** -0.5, window=window)


@pytest.mark.parametrize("scale", [1.0, -0.5])
@pytest.mark.parametrize("lengths,q_len,heads,rep,dim,group,window,dtype", FORMS)
def test_prompt_sharp_scores(lengths, q_len, heads, rep, dim, group, window, dtype, scale):
    """Scores of both signs, hundreds apart: the running maximum starts low and rises by much."""
    import bit_affine_quantized_qmv_amd as q
    s = Setup(lengths, heads, dim, group, 16, dtype, seed=dim + q_len)
    dev = s.len_dev.device
    queries = 8 * _rows((len(lengths), q_len, heads * rep, dim), dtype, 79, loud=False)
    y = q.kv_attend(queries.to(dev), s.cache, s.table, s.len_dev, scale=scale, window=window)
    torch.cuda.synchronize()
    s.check(y, queries, scale, window=window)
