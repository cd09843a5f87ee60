"""The bits that attention keeps: outputs within the roundings that each form states, where few
tokens are seen (the codes' term far larger than the output), and where most of the weight is on
one token and the output is what many small weights leave."""
import numpy as np
import pytest
import torch

from kv_precise import precise_reference
from qmm_testlib import TORCH_DTYPE, require_gpu, values
from test_gpu_kv_cache import _rows

pytestmark = pytest.mark.gpu


def attend(k, v, queries, group, dtype, scale, window=0, page=64):
    """y [q_len, q_heads, dim] of one sequence whose rows are k and v."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    n, heads, dim = k.shape
    blocks = -(-n // page)
    cache = q.kv_cache(blocks, page, heads, dim, group, dtype, dev)
    q.kv_append(cache, k.to(dev), v.to(dev), torch.arange(n, dtype=torch.int32, device=dev))
    table = torch.arange(blocks, dtype=torch.int32, device=dev)[None]
    y = q.kv_attend(queries[None].to(dev), cache, table, torch.tensor([n], dtype=torch.int32, device=dev), scale=scale,
                    window=window)
    torch.cuda.synchronize()
    return values(y[0])


def check(y, k, v, queries, group, dtype, scale, prompt, window=0):
    ref, tol = precise_reference(queries, k, v, k.shape[0], group, dtype, scale, prompt, window=window)
    err = np.abs(y - ref)
    assert (err <= tol).all(), "worst %.3g of the bound at %s" % (
        (err / tol).max(), np.unravel_index((err / tol).argmax(), err.shape))


@pytest.mark.parametrize("length,q_len,rep,dim,group,window,dtype,prompt", [
    (1, 1, 4, 128, 64, 0, "bf16", False), (2, 1, 4, 64, 32, 0, "fp16", False), (5, 5, 3, 64, 64, 0, "bf16", False),
    (7, 2, 2, 256, 128, 0, "fp16", False), (700, 4, 4, 128, 128, 3, "bf16", False), (700, 4, 4, 128, 64, 3, "fp16", False),
    (140, 140, 2, 128, 64, 3, "bf16", True), (140, 140, 2, 128, 32, 3, "fp16", True),
    (520, 520, 2, 64, 32, 2, "fp16", True), (520, 520, 2, 256, 64, 2, "bf16", True)])
def test_few_tokens_keep_the_stated_bits(length, q_len, rep, dim, group, window, dtype, prompt):
    """Values of both signs, much smaller than their groups' span in most elements."""
    k, v = (_rows((length, 1, dim), dtype, seed) for seed in (1, 2))
    queries = _rows((q_len, rep, dim), dtype, 3, loud=False)
    scale = dim ** -0.5
    y = attend(k, v, queries, group, dtype, scale, window)
    check(y, k, v, queries, group, dtype, scale, prompt, window)


@pytest.mark.parametrize("length,q_len,rep,dim,group,window,dtype,prompt", [
    (1, 1, 4, 128, 64, 0, "bf16", False), (1, 1, 4, 128, 64, 0, "fp16", False), (5, 5, 4, 128, 64, 0, "bf16", False),
    (5, 5, 4, 64, 32, 0, "fp16", False), (700, 4, 4, 128, 64, 3, "bf16", False), (300, 1, 3, 256, 64, 0, "bf16", False),
    (140, 140, 2, 128, 64, 3, "bf16", True), (140, 140, 2, 128, 128, 3, "fp16", True),
    (520, 520, 2, 64, 32, 2, "bf16", True), (520, 520, 2, 256, 128, 2, "fp16", True)])
def test_scores_near_zero_keep_the_stated_bits(length, q_len, rep, dim, group, window, dtype, prompt):
    """As above with weights that are nearly equal, where the bound is that of the operands."""
    k, v = (_rows((length, 1, dim), dtype, seed) for seed in (1, 2))
    queries = _rows((q_len, rep, dim), dtype, 3, loud=False) / 64
    scale = dim ** -0.5
    y = attend(k, v, queries, group, dtype, scale, window)
    check(y, k, v, queries, group, dtype, scale, prompt, window)


def dominated(n, dim, dtype, size, gap, seed):
    """Keys, values and a query direction: token 0 has the value 0 and a score `gap` above the
    others', whose values are size * (0.5 + a normal number)."""
    g = torch.Generator().manual_seed(seed)
    direction = torch.randn(dim, generator=g)
    k = 0.05 * torch.randn(n, 1, dim, generator=g)
    k[0, 0] = direction * (gap * dim ** 0.5 / direction.square().sum())
    v = size * (0.5 + torch.randn(n, 1, dim, generator=g))
    v[0] = 0.0
    return k.to(TORCH_DTYPE[dtype]), v.to(TORCH_DTYPE[dtype]), direction


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,dim,group,size,gap", [
    (8192, 64, 32, 1.0, 16.5), (8192, 128, 64, 0.005, 8.0), (8192, 128, 128, 0.02, 12.0), (3000, 256, 64, 1.0, 18.0),
    (131071, 128, 64, 1.0, 16.5), (131071, 64, 64, 0.02, 12.0)])
def test_small_weights_count_in_single_tokens(n, dim, group, size, gap, dtype):
    k, v, direction = dominated(n, dim, dtype, size, gap, n + dim)
    queries = (direction + 0.05 * torch.randn(1, 2, dim, generator=torch.Generator().manual_seed(4))).to(k.dtype)
    scale = dim ** -0.5
    y = attend(k, v, queries, group, dtype, scale)
    check(y, k, v, queries, group, dtype, scale, False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,q_len,rep,dim,group,size,gap", [
    (3000, 64, 4, 128, 64, 1.0, 18.0), (8192, 64, 4, 128, 32, 0.02, 14.0), (2500, 260, 4, 64, 64, 1.0, 19.0),
    (2500, 260, 4, 256, 128, 1.0, 16.5)])
def test_small_weights_count_in_prompts(n, q_len, rep, dim, group, size, gap, dtype):
    k, v, direction = dominated(n, dim, dtype, size, gap, n + dim)
    queries = (direction + 0.05 * torch.randn(q_len, rep, dim, generator=torch.Generator().manual_seed(4))).to(k.dtype)
    scale = dim ** -0.5
    y = attend(k, v, queries, group, dtype, scale)
    check(y, k, v, queries, group, dtype, scale, True)
