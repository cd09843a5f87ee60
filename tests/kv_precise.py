"""Reference of the attention forms with the bound of the roundings they state, term by term, in
float64 on the CPU (kv_testlib has the definition's codec; its bound allows more)."""
from __future__ import annotations

import numpy as np

from kv_testlib import cached_parts, half_ulp
from qmm_testlib import values

# Float32 arithmetic of one token's weight and of the sums over tokens: at most 256 roundings of
# 2^-24 in a row, for the sums relative to their terms, for a score relative to its own terms.
F32 = 2.0 ** -16
# Operands of the second product, two bfloat16 parts each.  Single tokens: p s_jg, its leading
# bits cut off, the rest rounded: 2^-16 of it, with exact codes.  Prompts: V (cut off 2^-16, in
# fp16 calls rounded 2^-17), p (rounded, 2^-17), and the product of the two rests left out
# (2^-7 or 2^-8 of V by 2^-8 of p): below 2^-14, in fp16 calls 2^-15, of |p v|.
SINGLE = 2.0 ** -16
PROMPT = {"bf16": 2.0 ** -14, "fp16": 2.0 ** -15}


def precise_reference(q, k, v, length, group, dtype, scale, prompt, causal=True, window=0):
    """One sequence, as kv_testlib.attend_reference: (out, tol) float64 [q_len, q_heads, d].

    With e_j the relative error of token j's weight, the output moves by sum w_j e_j v_j - out
    sum w_j e_j at most."""
    q_len, q_heads, d = q.shape
    rep = q_heads // k.shape[1]
    qv = values(q)
    out, tol = np.zeros((q_len, q_heads, d)), np.zeros((q_len, q_heads, d))
    ks, kc, kb = cached_parts(k, group, dtype)
    vs, vc, vb = cached_parts(v, group, dtype)
    kk, vv, codes = ks * kc + kb, vs * vc + vb, vs * vc
    k_size, v_size = ks * kc + np.abs(kb), codes + np.abs(vb)
    j = np.arange(length)
    for i in range(q_len):
        p = length - q_len + i
        see = (j <= p) if causal else np.ones(length, bool)
        if window:
            see = see & (j > p - window)
        if not see.any():
            continue
        see = slice(int(see.argmax()), int(see.argmax() + see.sum()))
        for h in range(q_heads):
            g = h // rep
            s = scale * (kk[see, g] @ qv[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv[see, g]
            e = w * (F32 * (1 + abs(scale) * (k_size[see, g] @ np.abs(qv[i, h]))))
            operands = PROMPT[dtype] * (w @ np.abs(vv[see, g])) if prompt else SINGLE * (w @ codes[see, g])
            tol[i, h] = operands + e @ v_size[see, g] + np.abs(out[i, h]) * e.sum()
    return out, tol + half_ulp(np.abs(out) + tol, dtype)
