"""Products grouped by expert, and the expert layer for any number of tokens, against float64
references of their definitions."""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from kv_testlib import half_ulp
from qmm_testlib import TORCH_DTYPE, half_bits, require_gpu, values, words
from test_gpu_moe import stack

pytestmark = pytest.mark.gpu

# Float32 sums: a rounding per matrix step of 32 products and two per group, at most 2 * K / 32 in
# all, so below 2^-17 of the terms' sizes up to K = 2048; twice that for the steps inside an
# instruction.  Terms are s x q and b x, so sizes are |x| (s q + |b|).
F32 = 2.0 ** -16
OPERANDS = 2.0 ** -16        # h as two bfloat16 parts: leading bits, and the rest rounded


def parts(w, e):
    """(w, size) float64 [N, K] of expert e: s q + b and |s| q + |b|."""
    q = w.expert(e)
    dtype = "bf16" if q.scales.dtype == torch.bfloat16 else "fp16"
    codes = O.unpack(words(q.w_packed), w.bits, w.K).astype(np.float64)
    s, b = (np.repeat(values(t), w.group_size, 1) for t in (q.scales, q.biases))
    assert dtype in TORCH_DTYPE
    return s * codes + b, np.abs(s) * codes + np.abs(b)


def product(x, w, e):
    """x W_e^T and its bound, float64."""
    full, size = parts(w, e)
    return x @ full.T, F32 * (np.abs(x) @ size.T)


def check(y, ref, tol):
    err = np.abs(values(y) - ref)
    assert (err <= tol).all(), "worst %.3g of the bound at %s" % ((err / np.maximum(tol, 1e-300)).max(),
                                                                 np.unravel_index((err - tol).argmax(), err.shape))


def rounded(ref, tol, dtype):
    return tol + half_ulp(np.abs(ref) + tol, dtype)


def offsets_of(counts, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32)


GROUPED = [
    # rows of each expert, N, K, bits, group, dtype
    ([1], 64, 128, 4, 64, "bf16"),
    ([1], 1, 32, 8, 32, "fp16"),                                   # one output
    ([5, 0, 16, 17, 33, 1], 100, 160, 4, 32, "fp16"),              # K and N inside a step and a tile
    ([31, 32, 0, 64, 65], 257, 384, 4, 64, "bf16"),
    ([40, 3, 0, 90], 130, 1408, 4, 128, "bf16"),                   # groups that are not whole words of scales
    ([100, 70], 300, 256, 8, 32, "bf16"),
    ([7, 200], 48, 448, 8, 64, "fp16"),
    ([129, 64, 3], 513, 384, 8, 128, "bf16"),
    ([20, 150], 70, 96, 2, 32, "bf16"),
    ([3, 66], 260, 192, 3, 64, "fp16"),
    ([80, 1], 33, 384, 5, 128, "bf16"),
    ([9, 100], 128, 224, 6, 32, "fp16"),
    ([2] * 512, 24, 64, 4, 32, "bf16"),                            # every expert there can be
    ([700], 96, 2048, 4, 64, "fp16"),                              # one expert
]


@pytest.mark.parametrize("counts,n,k,bits,group,dtype", GROUPED)
def test_grouped_matches_float64(counts, n, k, bits, group, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    w = stack(n, k, group, bits, dtype, len(counts), 10 * k + n, dev)
    rows = sum(counts)
    x = synth.normal_x((rows, k), dtype, seed=rows)
    offsets = offsets_of(counts)
    y = q.grouped_qmm(x.to(dev), w, offsets.to(dev))
    assert torch.equal(y, q.grouped_qmm(x.to(dev), w, offsets.to(dev)))
    xv = values(x)
    for e, c in enumerate(counts):
        if c:
            mine = slice(int(offsets[e]), int(offsets[e + 1]))
            ref, tol = product(xv[mine], w, e)
            check(y[mine], ref, rounded(ref, tol, dtype))


def padded(w, dev):
    """The same weights inside larger tensors: rows of NaN scales, odd alignment of scales."""
    import bit_affine_quantized_qmv_amd as q
    e, n, k = w.w_packed.shape
    codes = torch.full((e, n + 3, k + (-k) % 4 + 4), -1, dtype=torch.int32, device=dev)
    sb = [torch.full((e, n + 3, w.scales.shape[2] + 2), float("nan"), dtype=w.scales.dtype, device=dev) for _ in range(2)]
    codes[:, :n, :k] = w.w_packed
    sb[0][:, :n, 1:-1], sb[1][:, :n, 1:-1] = w.scales, w.biases
    return q.ExpertWeights(codes[:, :n, :k], sb[0][:, :n, 1:-1], sb[1][:, :n, 1:-1], w.N, w.K, w.group_size, w.bits)


@pytest.mark.parametrize("bits,group", [(4, 32), (4, 64), (8, 64), (4, 128), (6, 32), (3, 64)])
def test_grouped_strides_and_rows_of_nobody(bits, group):
    """Stacks, x and y inside larger tensors, first and last rows that belong to no expert."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    n, k, counts, dtype = 100, 7 * 128, [3, 40, 0, 9], "bf16"
    w = stack(n, k, group, bits, dtype, 4, 1, dev)
    rows = sum(counts) + 10
    big = torch.full((rows, k + 16), float("nan"), dtype=torch.bfloat16)
    big[:, 8:-8] = synth.normal_x((rows, k), dtype, seed=1)
    big[:4], big[-6:] = float("nan"), float("nan")
    out = torch.full((rows, n + 5), 7.0, dtype=torch.bfloat16, device=dev)
    offsets = offsets_of(counts, 4)
    q.grouped_qmm(big.to(dev)[:, 8:-8], padded(w, dev), offsets.to(dev), out=out[:, 2:2 + n])
    assert (out[:, :2] == 7.0).all() and (out[:, 2 + n:] == 7.0).all()
    assert (out[:4] == 7.0).all() and (out[-6:] == 7.0).all()
    for e, c in enumerate(counts):
        if c:
            mine = slice(int(offsets[e]), int(offsets[e + 1]))
            ref, tol = product(values(big[mine, 8:-8]), w, e)
            check(out[mine, 2:2 + n], ref, rounded(ref, tol, dtype))


def test_grouped_offsets_out_of_order():
    """Offsets outside the rows and descending ones: each row goes to one expert at most."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    w = stack(32, 64, 32, 4, "bf16", 4, 1, dev)
    x = synth.normal_x((50, 64), "bf16", seed=1)
    for given, taken in (([-5, 20, 10, 30, 99], [(0, 0, 20), (2, 20, 30), (3, 30, 50)]),
                         ([40, 10, 5, 45, 2 ** 31 - 1], [(2, 40, 45), (3, 45, 50)]),
                         ([-2 ** 31, -1, -1, 0, 0], []), ([60, 70, 80, 90, 100], [])):
        y = q.grouped_qmm(x.to(dev), w, torch.tensor(given, dtype=torch.int32, device=dev))
        want = torch.zeros_like(y)
        for e, a, b in taken:
            want[a:b] = q.grouped_qmm(x[a:b].to(dev), w, torch.tensor([0] * (e + 1) + [b - a] * (4 - e), dtype=torch.int32,
                                                                     device=dev))
        assert torch.equal(y, want)


def test_grouped_rows_are_the_same_in_tiles_of_any_height():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    for bits, group in ((4, 32), (4, 64), (4, 128), (8, 32), (8, 128), (6, 64)):
        w = stack(200, 384, group, bits, "bf16", 2, 1, dev)
        x = synth.normal_x((190, 384), "bf16", seed=1).to(dev)
        tall = q.grouped_qmm(x, w, torch.tensor([0, 100, 190], dtype=torch.int32, device=dev))
        low = q.grouped_qmm(x[90:150], w, torch.tensor([0, 10, 60], dtype=torch.int32, device=dev))
        assert torch.equal(tall[90:150], low)


def test_grouped_rows_are_the_same_in_tiles_of_sixteen():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    for bits, group in ((4, 32), (4, 64), (4, 128), (8, 32), (8, 128), (6, 64)):
        w = stack(200, 384, group, bits, "fp16", 2, 1, dev)
        x = synth.normal_x((190, 384), "fp16", seed=1).to(dev)
        tall = q.grouped_qmm(x, w, torch.tensor([0, 100, 190], dtype=torch.int32, device=dev))
        for counts in ((1, 15), (16, 0), (10, 6), (0, 1)):
            rows = x[100 - counts[0]:100 + counts[1]]
            low = q.grouped_qmm(rows, w, torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device=dev))
            assert torch.equal(tall[100 - counts[0]:100 + counts[1]], low), (bits, group, counts)


def test_grouped_rows_are_their_own():
    """A row's result is the same in any company, NaN rows aside."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    w = stack(70, 320, 64, 8, "fp16", 3, 1, dev)
    x = synth.normal_x((90, 320), "fp16", seed=1).to(dev)
    one = q.grouped_qmm(x, w, torch.tensor([0, 30, 31, 90], dtype=torch.int32, device=dev))
    x[40] = float("nan")
    x[50] = float("inf")
    two = q.grouped_qmm(x, w, torch.tensor([0, 30, 31, 90], dtype=torch.int32, device=dev))
    keep = [r for r in range(90) if r not in (40, 50)]
    assert torch.equal(one[keep], two[keep]) and not torch.isfinite(two[[40, 50]]).any()
    few = q.grouped_qmm(x[35:37], w, torch.tensor([0, 0, 0, 2], dtype=torch.int32, device=dev))
    assert torch.equal(few, one[35:37])
    assert q.grouped_qmm(x[:0], w, torch.zeros(4, dtype=torch.int32, device=dev)).shape == (0, 70)


def test_grouped_agrees_with_qmm_t_of_exact_weights():
    """Against the library's own product where both are exact: codes as weights."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    w = stack(128, 256, 64, 4, "bf16", 2, 1, dev)
    one, zero = torch.ones_like(w.scales), torch.zeros_like(w.biases)
    w = q.ExpertWeights(w.w_packed, one, zero, w.N, w.K, w.group_size, w.bits)
    x = torch.randint(-4, 5, (130, 256), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    y = q.grouped_qmm(x, w, torch.tensor([0, 60, 130], dtype=torch.int32, device=dev))
    assert torch.equal(y[:60], q.qmm_t(x[:60], w.expert(0))) and torch.equal(y[60:], q.qmm_t(x[60:], w.expert(1)))


# ---------------------------------------------------------------- the layer

def reference(x, router, gate, up, down, top_k, renormalize, dtype):
    xv, rv = values(x), values(router)
    tokens = xv.shape[0]
    y, tol = np.zeros((tokens, gate.K)), np.zeros((tokens, gate.K))
    chosen = np.argsort(-rv, axis=1, kind="stable")[:, :top_k]
    p = np.exp(rv - rv.max(1, keepdims=True))
    picked = np.take_along_axis(p, chosen, 1)
    share = picked / (picked if renormalize else p).sum(1, keepdims=True)
    for e in range(gate.num_experts):
        t, i = np.nonzero(chosen == e)
        if not len(t):
            continue
        (g, dg), (u, du) = product(xv[t], gate, e), product(xv[t], up, e)
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        h = silu * u
        # |silu'| <= 1.1; a few float32 operations on each factor
        dh = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 2.0 ** -18 * np.abs(h)
        dh = dh + OPERANDS * (np.abs(h) + dh)
        full, size = parts(down, e)
        s = share[t, i][:, None]
        np.add.at(y, t, s * (h @ full.T))
        np.add.at(tol, t, s * (dh @ np.abs(full).T + F32 * (np.abs(h) @ size.T)) * (1 + F32))
    return y, rounded(y, tol, dtype)


LAYERS = [
    # tokens, hidden, inter, experts, top_k, (bits, group) of gate/up, of down, dtype
    (1, 128, 96, 3, 1, (4, 32), (8, 32), "fp16"),
    (33, 256, 128, 8, 2, (4, 64), (4, 64), "bf16"),
    (70, 320, 704, 6, 4, (4, 64), (6, 64), "bf16"),
    (200, 352, 224, 20, 4, (8, 32), (8, 32), "bf16"),
    (150, 512, 256, 4, 3, (4, 128), (4, 128), "fp16"),
    (90, 256, 384, 70, 8, (8, 64), (8, 128), "bf16"),
    (100, 192, 160, 2, 2, (8, 64), (4, 32), "fp16"),          # every token through every expert
    (40, 384, 640, 5, 2, (2, 128), (3, 32), "bf16"),
    (45, 224, 192, 6, 2, (3, 32), (5, 64), "fp16"),
    (64, 32, 32, 512, 32, (4, 32), (4, 32), "bf16"),          # the limits of experts and top_k
    (300, 640, 1152, 3, 1, (6, 128), (8, 128), "fp16"),
]


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,first,second,dtype", LAYERS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_layer_matches_float64(tokens, hidden, inter, experts, top_k, first, second, dtype, renormalize):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gate = stack(inter, hidden, first[1], first[0], dtype, experts, 100 + tokens, dev)
    up = stack(inter, hidden, first[1], first[0], dtype, experts, 2000 + tokens, dev)
    down = stack(hidden, inter, second[1], second[0], dtype, experts, 4000 + tokens, dev)
    x = synth.normal_x((tokens, hidden), dtype, seed=tokens)
    router = (1.5 * synth.normal_x((tokens, experts), "bf16", seed=tokens + 1).float()).to(TORCH_DTYPE[dtype])
    ws = q.moe_prompt_workspace(x.to(dev), gate, top_k)
    ws.fill_(float("nan"))
    y = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, top_k, renormalize=renormalize, workspace=ws)
    again = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, top_k, renormalize=renormalize)
    ref, tol = reference(x, router, gate, up, down, top_k, renormalize, dtype)
    check(y, ref, tol)
    assert torch.equal(y, again)


LONG = [
    # few rows of long ones: the second product's columns are shared out
    (1, 64, 2080, 3, 1, (4, 32), (4, 32), "bf16"),            # 65 groups: two runs of 32 and one more
    (5, 160, 2048, 4, 2, (8, 32), (8, 32), "fp16"),
    (9, 96, 4160, 2, 1, (4, 32), (4, 64), "fp16"),
    (40, 64, 4160, 2, 2, (4, 32), (8, 64), "bf16"),
    (130, 128, 8320, 1, 1, (4, 64), (4, 128), "bf16"),
    (3, 32, 8192, 2, 1, (4, 32), (6, 128), "fp16"),
    (20, 64, 3200, 2, 1, (3, 32), (3, 32), "bf16"),
]


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,first,second,dtype", LONG)
def test_layer_of_few_rows_and_long_ones(tokens, hidden, inter, experts, top_k, first, second, dtype):
    test_layer_matches_float64(tokens, hidden, inter, experts, top_k, first, second, dtype, True)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32), (6, 128)])
@pytest.mark.parametrize("x_size,down_std", [(30.0, 1e-4), (0.0003, 1000.0)])
def test_layer_hidden_values_of_any_size(x_size, down_std, bits, group, dtype):
    """h around 1e5 and 6e-6."""
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    tokens, hidden, inter, experts, top_k = 40, 128, 256, 4, 2
    gate, up = (stack(inter, hidden, group, bits, dtype, experts, s, dev, std=1.0) for s in (1, 500))
    down = stack(hidden, inter, group, bits, dtype, experts, 900, dev, std=down_std)
    x = (x_size * synth.normal_x((tokens, hidden), "bf16", seed=1).float()).to(TORCH_DTYPE[dtype])
    router = synth.normal_x((tokens, experts), dtype, seed=2)
    y = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, top_k)
    ref, tol = reference(x, router, gate, up, down, top_k, True, dtype)
    assert (np.abs(ref).max() < 60000) and (np.abs(ref).max() > 1e-3)
    check(y, ref, tol)


def test_layer_ties_masks_and_values_that_are_not_finite():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    dtype, tokens, experts = "bf16", 50, 100
    gate, up = (stack(64, 128, 64, 4, dtype, experts, s, dev) for s in (1, 500))
    down = stack(128, 64, 64, 4, dtype, experts, 900, dev)
    x = synth.normal_x((tokens, 128), dtype, seed=1)
    router = synth.normal_x((tokens, experts), dtype, seed=3)
    router[0] = 0.0                                                       # all equal: experts 0, 1, 2
    router[1] = 0.0
    router[1, 50:] = 1.0                                                  # experts 50, 51, 52
    router[2] = torch.finfo(torch.bfloat16).min                           # a mask of the lowest value
    router[3] = -float("inf")
    router[3, [7, 70, 99]] = 0.5                                          # masked experts get nothing
    router[4] = 0.0
    router[4, 3] = -0.0
    router[5] = torch.finfo(torch.bfloat16).min
    router[5, 42] = 2.0                                                   # one open expert, two of weight 0
    y = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, 3)
    ref, tol = reference(x, router, gate, up, down, 3, True, dtype)
    check(y, ref, tol)
    small = q.moe(x[:32].to(dev), router[:32].to(dev), gate, up, down, 3)
    check(small, ref[:32], tol[:32])
    router[10, 6] = float("nan")
    x[20, 5] = float("inf")
    z = q.moe_prompt(x.to(dev), router.to(dev), gate, up, down, 3)
    keep = [t for t in range(tokens) if t not in (10, 20)]
    assert torch.equal(z[keep], y[keep])
    assert torch.isnan(z[10].float()).all() and not torch.isfinite(z[20].float()).any()


@pytest.mark.parametrize("bits,gs", [(4, 32), (8, 64), (6, 32), (4, 128)])
def test_layer_padded_stacks_and_strided_rows(bits, gs):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    dtype, tokens, hidden, inter, experts = "bf16", 77, 7 * 128, 384, 6
    gate, up = (stack(inter, hidden, gs, bits, dtype, experts, s, dev) for s in (1, 500))
    down = stack(hidden, inter, gs, bits, dtype, experts, 900, dev)
    big = torch.full((tokens, hidden + 16), float("nan"), dtype=torch.bfloat16)
    big[:, 8:-8] = synth.normal_x((tokens, hidden), dtype, seed=1)
    router = torch.full((tokens, experts + 3), float("nan"), dtype=torch.bfloat16)
    router[:, 1:-2] = synth.normal_x((tokens, experts), dtype, seed=2)
    out = torch.full((tokens, hidden + 5), 7.0, dtype=torch.bfloat16, device=dev)
    q.moe_prompt(big.to(dev)[:, 8:-8], router.to(dev)[:, 1:-2], padded(gate, dev), padded(up, dev), padded(down, dev), 3,
                 out=out[:, 1:1 + hidden])
    ref, tol = reference(big[:, 8:-8], router[:, 1:-2], gate, up, down, 3, True, dtype)
    check(out[:, 1:1 + hidden], ref, tol)
    assert (out[:, 0] == 7.0).all() and (out[:, 1 + hidden:] == 7.0).all()


def test_layer_another_stream_and_graph_replays():
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gate, up = (stack(256, 512, 64, 4, "bf16", 16, s, dev) for s in (1, 500))
    down = stack(512, 256, 64, 4, "bf16", 16, 900, dev)
    x = synth.normal_x((111, 512), "bf16", seed=1).to(dev)
    router = synth.normal_x((111, 16), "bf16", seed=2).to(dev)
    offsets = torch.tensor([0] + [20] * 15 + [111], dtype=torch.int32, device=dev)
    want, want2 = q.moe_prompt(x, router, gate, up, down, 4), q.grouped_qmm(x, gate, offsets)
    ws, ws2 = q.moe_prompt_workspace(x, gate, 4), q.grouped_workspace(x, gate)
    out, out2 = torch.empty_like(want), torch.empty_like(want2)

    def both():
        q.moe_prompt(x, router, gate, up, down, 4, out=out, workspace=ws)
        q.grouped_qmm(x, gate, offsets, out=out2, workspace=ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(out2, want2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for i in range(4):
        if i == 2:                                                       # new routing, new offsets
            router.copy_(router.flip(1))
            offsets.copy_(torch.tensor([0, 100] + [111] * 15, dtype=torch.int32))
            want, want2 = q.moe_prompt(x, router, gate, up, down, 4), q.grouped_qmm(x, gate, offsets)
        out.zero_()
        out2.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(out2, want2)
        q.moe_prompt(x[:40], router[:40], gate, up, down, 4, workspace=ws)      # eager work between replays
        torch.cuda.synchronize()
    assert q.moe_prompt(x[:0], router[:0], gate, up, down, 4).shape == (0, 512)
