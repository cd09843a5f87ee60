"""The expert layer where a row of the second product is cut into several workgroups' stretches
and each wave takes whole tiles of them, against the float64 reference and its bounds."""
import pytest
import torch

import synth
from qmm_testlib import TORCH_DTYPE, require_gpu
from test_gpu_moe import check, reference

pytestmark = pytest.mark.gpu


class Cycle:
    """A stack whose expert e is matrix e % len(matrices), as the reference wants it."""

    def __init__(self, matrices):
        self.m = matrices
        for name in ("N", "K", "bits", "group_size"):
            setattr(self, name, getattr(matrices[0], name))

    def expert(self, e):
        return self.m[e % len(self.m)]


@pytest.mark.parametrize("tokens,top_k,dtype", [(3, 8, "bf16"), (17, 2, "fp16")])
def test_moe_long_second_product(tokens, top_k, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    hidden, inter, experts = 2048, 6208, 24
    gen = torch.Generator(device=dev).manual_seed(3)

    def matrices(n, k):
        return [q.quantize(0.05 * torch.randn(n, k, generator=gen, device=dev), 64, 4, TORCH_DTYPE[dtype])
                for _ in range(2)]

    roles = [matrices(inter, hidden), matrices(inter, hidden), matrices(hidden, inter)]
    gate, up, down = (q.ExpertWeights.stack([m[e % 2] for e in range(experts)]) for m in roles)
    x = synth.normal_x((tokens, hidden), dtype, seed=tokens)
    router = (1.5 * synth.normal_x((tokens, experts), "bf16", seed=tokens + 1).float()).to(TORCH_DTYPE[dtype])
    y = q.moe(x.to(dev), router.to(dev), gate, up, down, top_k)
    torch.cuda.synchronize()

    ref, tol = reference(x, router, *(Cycle(m) for m in roles), top_k, True, dtype)
    check(y, ref, tol)
