"""The mixture-of-experts layer against a float64 reference of its definition."""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from kv_testlib import half_ulp
from qmm_testlib import TORCH_DTYPE, half_bits, require_gpu, upload_oracle_weight, values, words

pytestmark = pytest.mark.gpu

ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}      # relative error of one rounding, at most
SUBNORMAL = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
# Float32 sums of at most a few thousand terms on the matrix cores: far below 2^-18 of the sum
# of the terms' magnitudes (2^-24 per step, errors of both signs).
F32 = 2.0 ** -18


def stack(n, k, gs, bits, dtype, count, seed, dev, std=0.05):
    import bit_affine_quantized_qmv_amd as q
    ws = [upload_oracle_weight(O.quantize(synth.normal_weight(n, k, std, seed=seed + e).numpy(), gs, bits, dtype), dev)
          for e in range(count)]
    return q.ExpertWeights.stack(ws)


def dense(w, e, dtype):
    q = w.expert(e)
    codes = O.unpack(words(q.w_packed), w.bits, w.K)
    return O.dequant(codes, half_bits(q.scales), half_bits(q.biases), w.group_size, dtype)


def reference(x, router, gate, up, down, top_k, renormalize, dtype):
    xv, rv = values(x), values(router)
    tokens = xv.shape[0]
    y, tol = np.zeros((tokens, gate.K)), np.zeros((tokens, gate.K))
    mats = {}
    for t in range(tokens):
        chosen = np.argsort(-rv[t], kind="stable")[:top_k]
        p = np.exp(rv[t] - rv[t].max())
        p = p / (p[chosen].sum() if renormalize else p.sum())
        for e in chosen:
            if e not in mats:
                mats[e] = [dense(w, int(e), dtype) for w in (gate, up, down)]
            wg, wu, wd = mats[e]
            g, u = wg @ xv[t], wu @ xv[t]
            dg, du = F32 * (np.abs(wg) @ np.abs(xv[t])), F32 * (np.abs(wu) @ np.abs(xv[t]))
            silu = g / (1 + np.exp(-g))
            h = p[e] * silu * u
            # |silu'| <= 1.1; a few float32 operations on each factor
            dh = p[e] * (1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du) + 2.0 ** -18 * np.abs(h)
            dh = dh + ROUND[dtype] * (np.abs(h) + dh) + SUBNORMAL[dtype]
            y[t] += wd @ h
            tol[t] += np.abs(wd) @ dh + F32 * (np.abs(wd) @ np.abs(h))
    return y, tol + half_ulp(np.abs(y) + tol, dtype)


def check(y, ref, tol, rows=None):
    yv = values(y)
    if rows is not None:
        yv, ref, tol = yv[rows], ref[rows], tol[rows]
    err = np.abs(yv - ref)
    assert (err <= tol).all(), "worst %.3g of the bound" % (err / tol).max()


CASES = [
    # tokens, hidden, inter, experts, top_k, (bits, group) of gate/up, of down, dtype
    (1, 2048, 1024, 8, 2, (4, 64), (4, 64), "bf16"),
    (1, 128, 96, 3, 1, (4, 32), (8, 32), "fp16"),
    (5, 320, 704, 16, 4, (4, 64), (6, 64), "bf16"),
    (16, 1408, 704, 20, 4, (8, 32), (8, 32), "bf16"),
    (17, 512, 256, 40, 3, (4, 128), (4, 128), "fp16"),
    (32, 256, 384, 70, 8, (8, 64), (8, 128), "bf16"),
    (32, 192, 160, 2, 2, (8, 64), (4, 32), "fp16"),          # every token through every expert
    (7, 4096, 224, 4, 2, (4, 128), (4, 32), "bf16"),
    (3, 256, 128, 5, 2, (2, 64), (2, 32), "bf16"),
    (18, 224, 192, 6, 2, (3, 32), (3, 64), "fp16"),
    (2, 384, 256, 4, 4, (5, 128), (5, 64), "bf16"),
    (20, 384, 256, 4, 1, (6, 64), (6, 128), "bf16"),
    (6, 32, 32, 512, 32, (4, 32), (4, 32), "bf16"),          # the limits of experts and top_k
    (4, 8192, 64, 2, 1, (8, 128), (8, 32), "fp16"),
]


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,first,second,dtype", CASES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_moe_matches_float64(tokens, hidden, inter, experts, top_k, first, second, dtype, renormalize):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gate = stack(inter, hidden, first[1], first[0], dtype, experts, 100 + tokens, dev)
    up = stack(inter, hidden, first[1], first[0], dtype, experts, 2000 + tokens, dev)
    down = stack(hidden, inter, second[1], second[0], dtype, experts, 4000 + tokens, dev)
    x = synth.normal_x((tokens, hidden), dtype, seed=tokens)
    router = (1.5 * synth.normal_x((tokens, experts), "bf16", seed=tokens + 1).float()).to(TORCH_DTYPE[dtype])
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k, renormalize=renormalize)
    again = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k, renormalize=renormalize)
    torch.cuda.synchronize()
    ref, tol = reference(x, router, gate, up, down, top_k, renormalize, dtype)
    check(y, ref, tol)
    assert torch.equal(y, again)


def test_moe_ties_take_the_lower_expert_and_lowest_values_are_ordinary():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    dtype, tokens, experts = "bf16", 6, 100
    gate, up = (stack(64, 128, 64, 4, dtype, experts, s, dev) for s in (1, 500))
    down = stack(128, 64, 64, 4, dtype, experts, 900, dev)
    x = synth.normal_x((tokens, 128), dtype, seed=1)
    router = torch.zeros(tokens, experts, dtype=torch.bfloat16)          # all equal: experts 0, 1, 2
    router[1, 50:] = 1.0                                                  # experts 50, 51, 52
    router[2] = torch.finfo(torch.bfloat16).min                           # a mask of the lowest value
    router[3] = -float("inf")
    router[3, [7, 70, 99]] = 0.5                                          # masked experts get nothing
    router[4, 3] = -0.0
    router[5] = torch.finfo(torch.bfloat16).min
    router[5, 42] = 2.0                                                   # one open expert, two of weight 0
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, 3)
    torch.cuda.synchronize()
    ref, tol = reference(x, router, gate, up, down, 3, True, dtype)
    check(y, ref, tol)


def test_moe_nan_router_poisons_its_token_only():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gate, up = (stack(64, 128, 32, 4, "fp16", 8, s, dev) for s in (1, 500))
    down = stack(128, 64, 32, 4, "fp16", 8, 900, dev)
    x = synth.normal_x((4, 128), "fp16", seed=1)
    router = synth.normal_x((4, 8), "fp16", seed=2)
    clean = q.moe(x.to(dev), router.to(dev), gate, up, down, 2)
    router[1, 6] = float("nan")
    x[3, 5] = float("inf")
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, 2)
    torch.cuda.synchronize()
    assert torch.isnan(y[1].float()).all() and not torch.isfinite(y[3].float()).any()
    assert torch.equal(y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("bits,gs", [(4, 32), (8, 64), (6, 32), (3, 64)])
def test_moe_padded_stacks_and_strided_rows(bits, gs):
    """Expert stacks inside larger tensors (padded rows of NaN scales, odd scale alignment), x,
    the router and y as slices: nothing outside is read or written."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    dtype, tokens, hidden, inter, experts = "bf16", 9, 7 * 64, 192, 6

    def padded(w):
        words_pad = torch.full((experts, w.N + 3, w.w_packed.shape[2] + 8), -1, dtype=torch.int32, device=dev)
        words_pad = words_pad[:, :, :w.w_packed.shape[2] + (-w.w_packed.shape[2]) % 4 + 4].contiguous()
        sb = [torch.full((experts, w.N + 3, w.scales.shape[2] + 1), float("nan"), dtype=w.scales.dtype, device=dev)
              for _ in range(2)]
        words_pad[:, :w.N, :w.w_packed.shape[2]] = w.w_packed
        sb[0][:, :w.N, 1:] = w.scales
        sb[1][:, :w.N, 1:] = w.biases
        return q.ExpertWeights(words_pad[:, :w.N, :w.w_packed.shape[2]], sb[0][:, :w.N, 1:], sb[1][:, :w.N, 1:], w.N,
                               w.K, w.group_size, w.bits)

    gate, up = (stack(inter, hidden, gs, bits, dtype, experts, s, dev) for s in (1, 500))
    down = stack(hidden, inter, gs, bits, dtype, experts, 900, dev)
    big = torch.full((tokens, hidden + 16), float("nan"), dtype=torch.bfloat16)
    big[:, 8:-8] = synth.normal_x((tokens, hidden), dtype, seed=1)
    router = torch.full((tokens, experts + 3), float("nan"), dtype=torch.bfloat16)
    router[:, 1:-2] = synth.normal_x((tokens, experts), dtype, seed=2)
    out = torch.full((tokens, hidden + 5), 7.0, dtype=torch.bfloat16, device=dev)
    y = q.moe(big.to(dev)[:, 8:-8], router.to(dev)[:, 1:-2], padded(gate), padded(up), padded(down), 3,
              out=out[:, 1:1 + hidden])
    torch.cuda.synchronize()
    ref, tol = reference(big[:, 8:-8], router[:, 1:-2], gate, up, down, 3, True, dtype)
    check(y, ref, tol)
    assert (out[:, 0] == 7.0).all() and (out[:, 1 + hidden:] == 7.0).all()


def test_moe_another_stream_and_graph_replays():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gate, up = (stack(512, 1024, 64, 4, "bf16", 16, s, dev) for s in (1, 500))
    down = stack(1024, 512, 64, 4, "bf16", 16, 900, dev)
    x = synth.normal_x((11, 1024), "bf16", seed=1).to(dev)
    router = synth.normal_x((11, 16), "bf16", seed=2).to(dev)
    want = q.moe(x, router, gate, up, down, 4)
    ws = q.moe_workspace(x, gate, 4)
    ws.fill_(float("nan"))
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.moe(x, router, gate, up, down, 4, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.moe(x, router, gate, up, down, 4, out=out, workspace=ws)
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        q.moe(x[:2], router[:2], gate, up, down, 4, workspace=ws)    # eager work between replays
        torch.cuda.synchronize()
    assert q.moe(x[:0], router[:0], gate, up, down, 4).shape == (0, 1024)
