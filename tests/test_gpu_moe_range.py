"""The expert layer's hidden values far from one, of both types: the second product takes them
with float32's range and 16 bits, so outputs that are ordinary numbers come out."""
import numpy as np
import pytest
import torch

import synth
from kv_testlib import half_ulp
from qmm_testlib import TORCH_DTYPE, require_gpu, values
from test_gpu_moe import F32, check, dense, stack

pytestmark = pytest.mark.gpu

OPERANDS = 2.0 ** -16        # h as two bfloat16 parts, both rounded (2^-17)


def reference(x, router, gate, up, down, top_k, dtype):
    """As test_gpu_moe.reference, with h's two parts in place of one rounding to the type."""
    xv, rv = values(x), values(router)
    y, tol = np.zeros((xv.shape[0], gate.K)), np.zeros((xv.shape[0], gate.K))
    for t in range(xv.shape[0]):
        chosen = np.argsort(-rv[t], kind="stable")[:top_k]
        p = np.exp(rv[t] - rv[t].max())
        p = p / p[chosen].sum()
        for e in chosen:
            wg, wu, wd = (dense(w, int(e), dtype) for w in (gate, up, down))
            g, u = wg @ xv[t], wu @ xv[t]
            dg, du = F32 * (np.abs(wg) @ np.abs(xv[t])), F32 * (np.abs(wu) @ np.abs(xv[t]))
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = p[e] * silu * u
            dh = p[e] * (1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du) + F32 * np.abs(h)
            dh = dh + OPERANDS * (np.abs(h) + dh)
            y[t] += wd @ h
            tol[t] += np.abs(wd) @ dh + F32 * (np.abs(wd) @ np.abs(h))
    return y, tol + half_ulp(np.abs(y) + tol, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32), (6, 128)])
@pytest.mark.parametrize("x_size,down_std", [(30.0, 1e-4), (0.0003, 1000.0), (1.0, 0.05)])
def test_hidden_values_of_any_size(x_size, down_std, bits, group, dtype):
    """h around 1e5, 6e-6 and 1."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    tokens, hidden, inter, experts, top_k = 5, 128, 256, 4, 2
    wide = 1.0 if x_size != 1.0 else 0.1
    gate, up = (stack(inter, hidden, group, bits, dtype, experts, s, dev, std=wide) for s in (1, 500))
    down = stack(hidden, inter, group, bits, dtype, experts, 900, dev, std=down_std)
    x = (x_size * synth.normal_x((tokens, hidden), "bf16", seed=1).float()).to(TORCH_DTYPE[dtype])
    router = synth.normal_x((tokens, experts), dtype, seed=2)
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k)
    torch.cuda.synchronize()
    ref, tol = reference(x, router, gate, up, down, top_k, dtype)
    assert (np.abs(ref).max() < 60000) and (np.abs(ref).max() > 1e-3)
    check(y, ref, tol)
