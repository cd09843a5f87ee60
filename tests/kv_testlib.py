"""References of the cache and attention tests, in float64 on the CPU, from the definitions
(numpy; the codec comes from the oracle)."""
from __future__ import annotations

import numpy as np

import oracle as O
from qmm_testlib import values

HALF_ULP = {"bf16": 2.0 ** -9, "fp16": 2.0 ** -12}   # relative, of one rounding to the type
MIN_EXP = {"bf16": -133, "fp16": -24}                # exponent of the smallest subnormal


def half_ulp(x, dtype):
    """Half a unit in the last place of `dtype` at |x|."""
    bits = {"bf16": 8, "fp16": 11}[dtype]
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -200)))
    return 0.5 * 2.0 ** np.maximum(e - bits + 1, MIN_EXP[dtype])


def cached_parts(rows, group, dtype):
    """(s, c, b) in float64 [..., d] of the cached form of a bf16/fp16 tensor [..., d]."""
    flat = rows.reshape(-1, rows.shape[-1])
    q = O.quantize(flat.float().cpu().numpy(), group, 4, dtype)
    s, b = _f64(q["scales_bits"], dtype), _f64(q["biases_bits"], dtype)
    shape = tuple(rows.shape)
    return (np.repeat(s, group, 1).reshape(shape), q["codes"].astype(np.float64).reshape(shape),
            np.repeat(b, group, 1).reshape(shape))


def _f64(bits, dtype):
    if dtype == "fp16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def attend_reference(q, k, v, length, group, dtype, scale, causal, window):
    """One sequence: q [q_len, q_heads, d], k and v [length, heads, d] as appended (torch,
    in dtype).  Returns (out, tol) float64 [q_len, q_heads, d].

    tol bounds what the operator's stated roundings can do: p * s rounded once to dtype
    (relative half ulp of the code part of the sum, plus half the smallest subnormal for each
    of the `length` terms with codes up to 15, over a sum of at least 1), float32 scores and
    exponentials (2^-16 of the mean |v| per unit of the largest score is far above their
    2^-23 steps over a few hundred operations), and the final rounding."""
    q_len, q_heads, d = q.shape
    heads = k.shape[1]
    rep = q_heads // heads
    qv = values(q)
    out, tol = np.zeros((q_len, q_heads, d)), np.zeros((q_len, q_heads, d))
    if length == 0:
        return out, tol
    ks, kc, kb = cached_parts(k, group, dtype)
    vs, vc, vb = cached_parts(v, group, dtype)
    kk, vv = ks * kc + kb, vs * vc + vb
    j = np.arange(length)
    for i in range(q_len):
        p = length - q_len + i
        see = (j <= p) if causal else np.ones(length, bool)
        if window:
            see &= j > p - window
        if not see.any():
            continue
        for h in range(q_heads):
            g = h // rep
            s = scale * (kk[see, g] @ qv[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv[see, g]
            code_part = w @ (vs[see, g] * vc[see, g])
            size = abs(scale) * np.abs(kk[see, g]) @ np.abs(qv[i, h])
            tol[i, h] = (HALF_ULP[dtype] * code_part + see.sum() * 15 * 2.0 ** (MIN_EXP[dtype] - 1)
                         + 2.0 ** -16 * (1 + size.max()) * (w @ np.abs(vv[see, g])) + half_ulp(out[i, h], dtype))
    # the final rounding may sit on the next binade of a perturbed value
    return out, tol + half_ulp(np.abs(out) + tol, dtype) - half_ulp(out, dtype)
