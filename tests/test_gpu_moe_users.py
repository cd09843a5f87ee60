"""The expert layer where many tokens share an expert and its rows are long: the activations of up
to 16 of them pass through LDS in chunks of a few slots, shared by the waves of a tile.  Against
the float64 reference and its bounds."""
import pytest
import torch

import synth
from qmm_testlib import TORCH_DTYPE, require_gpu
from test_gpu_moe import check, reference
from test_gpu_moe_long import Cycle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,top_k", [(16, 4, 2), (32, 8, 2), (12, 2, 2)])
@pytest.mark.parametrize("bits,group", [(4, 128), (6, 128), (8, 128), (4, 64)])
@pytest.mark.parametrize("hidden,inter,dtype", [(512, 1024, "bf16"), (640, 2048, "fp16")])
def test_moe_many_users_of_an_expert(hidden, inter, bits, group, tokens, experts, top_k, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    gen = torch.Generator(device=dev).manual_seed(bits + tokens)

    def matrices(n, k):
        return [q.quantize(0.05 * torch.randn(n, k, generator=gen, device=dev), group, bits, TORCH_DTYPE[dtype])
                for _ in range(2)]

    roles = [matrices(inter, hidden), matrices(inter, hidden), matrices(hidden, inter)]
    gate, up, down = (q.ExpertWeights.stack([m[e % 2] for e in range(experts)]) for m in roles)
    x = synth.normal_x((tokens, hidden), dtype, seed=tokens)
    router = synth.normal_x((tokens, experts), "bf16", seed=tokens + 1).to(TORCH_DTYPE[dtype])
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k)
    again = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k)
    torch.cuda.synchronize()

    ref, tol = reference(x, router, *(Cycle(m) for m in roles), top_k, True, dtype)
    check(y, ref, tol)
    assert torch.equal(y, again)
