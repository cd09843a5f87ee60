"""CPU tests of the bounds that hold attention and the expert layer to the bits they state: the
arithmetic with two bfloat16 parts is inside them; one part, or fp16 parts where weights are
small, is not.  The arithmetic is modelled here, in float64 but for the operands' roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_precise import precise_reference
from kv_testlib import cached_parts, half_ulp
from qmm_testlib import TORCH_DTYPE, values
from test_gpu_kv_cache import _rows
from test_gpu_kv_precision import dominated


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TORCH_DTYPE[dtype]).double().numpy()


def cut(x):
    """Leading bfloat16 bits, the rest cut off."""
    b = x.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)
    return b.view(np.float32).astype(np.float64)


def two(x, first, dtype="bf16"):
    hi = first(x)
    return hi + rounded(x - hi, dtype)


OPERANDS = {"two": lambda x: two(x, cut), "one": lambda x: rounded(x, "bf16"),
            "fp16": lambda x: two(x, lambda v: rounded(v, "fp16"), "fp16")}


def attend_model(queries, k, v, group, dtype, scale, prompt, operand, window=0):
    """One kv head, causal; the first operand's roundings as `operand` says."""
    n, (q_len, q_heads, d) = k.shape[0], queries.shape
    ks, kc, kb = (a[:, 0] for a in cached_parts(k, group, dtype))
    vs, vc, vb = (a[:, 0] for a in cached_parts(v, group, dtype))
    kk, qv, out = ks * kc + kb, values(queries), np.zeros((q_len, q_heads, d))
    f = OPERANDS[operand]
    for i in range(q_len):
        hi = n - q_len + i + 1
        see = slice(max(0, hi - window) if window else 0, hi)
        for h in range(q_heads):
            s = scale * (kk[see] @ qv[i, h])
            p = np.exp(s - s.max())
            if prompt:
                acc = f(p) @ f(vs[see] * vc[see] + vb[see])
            else:
                acc = (f(p[:, None] * vs[see]) * vc[see]).sum(0) + p @ vb[see]
            out[i, h] = rounded(acc / p.sum(), dtype)
    return out


def outside(queries, k, v, group, dtype, prompt, operand, window=0):
    scale = k.shape[2] ** -0.5
    y = attend_model(queries, k, v, group, dtype, scale, prompt, operand, window)
    ref, tol = precise_reference(queries, k, v, k.shape[0], group, dtype, scale, prompt, window=window)
    return (np.abs(y - ref) > tol).any()


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("length,q_len,window", [(1, 1, 0), (5, 5, 0), (700, 4, 3)])
def test_attention_few_tokens_needs_both_parts(length, q_len, window, dtype, prompt):
    k, v = (_rows((length, 1, 128), dtype, seed) for seed in (1, 2))
    queries = _rows((q_len, 4, 128), dtype, 3, loud=False) / 64     # scores near zero: their errors are small
    assert not outside(queries, k, v, 64, dtype, prompt, "two", window)
    if length > 1:                           # (one token's p is 1)
        assert outside(queries, k, v, 64, dtype, prompt, "one", window)


@pytest.mark.parametrize("prompt,n,size,gap", [(False, 8192, 0.02, 12.0), (False, 3000, 1.0, 18.0),
                                               (True, 3000, 1.0, 18.0), (True, 2500, 1.0, 16.5)])
def test_attention_small_weights_need_the_range_of_bfloat16(prompt, n, size, gap):
    k, v, direction = dominated(n, 128, "fp16", size, gap, n)
    queries = direction.expand(1, 2, 128).to(k.dtype)
    assert not outside(queries, k, v, 64, "fp16", prompt, "two")
    assert outside(queries, k, v, 64, "fp16", prompt, "fp16")


@pytest.mark.parametrize("dtype,std,down_std,wrong", [("bf16", 1.0, 1.0, "one"), ("fp16", 1.0, 1.0, "one"),
                                                      ("fp16", 2.0 ** -18, 512.0, "fp16")])
def test_hidden_values_need_both_parts(dtype, std, down_std, wrong):
    """The second product of one expert, whose terms the bound of its tests takes with 2^-16."""
    w = down_std * torch.randn(64, 256, generator=torch.Generator().manual_seed(1))
    q = O.quantize(w.numpy(), 64, 4, dtype)
    wd = O.dequant(q["codes"], q["scales_bits"], q["biases_bits"], 64, dtype)
    h = std * torch.randn(256, generator=torch.Generator().manual_seed(2)).double().numpy()
    ref = wd @ h
    tol = (2.0 ** -16 + 2.0 ** -18) * (np.abs(wd) @ np.abs(h))
    tol = tol + half_ulp(np.abs(ref) + tol, dtype)

    def off(operand):
        return (np.abs(rounded(wd @ OPERANDS[operand](h), dtype) - ref) > tol).any()

    assert not off("two") and off(wrong)
