"""Settings of sampling that are not numbers, or outside of their ranges, mean what the header says."""
import pytest
import torch

from qmm_testlib import require_gpu

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.mark.parametrize("n", [5, 3000, 20000])
@pytest.mark.parametrize("settings", [
    dict(temperature=NAN), dict(temperature=-1.0), dict(top_p=NAN), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=NAN),
    dict(min_p=1.5), dict(top_k=1)])
def test_settings_that_leave_the_first_largest(settings, n):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    x = torch.randn(4, n, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    u = torch.tensor([0.0, 0.3, 0.9, 1.0])
    index, prob = q.sample(x.to(dev), u.to(dev), **settings)
    torch.cuda.synchronize()
    assert index.tolist() == [int((row == row.max()).nonzero()[0]) for row in x]
    assert prob.tolist() == [1.0] * 4


@pytest.mark.parametrize("settings", [dict(top_p=7.0), dict(min_p=-2.0), dict(top_k=-3), dict(top_k=10 ** 9)])
def test_settings_that_leave_everything(settings):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    x = torch.randn(6, 3000, generator=torch.Generator().manual_seed(1)).to(torch.float16).to(dev)
    u = torch.tensor([0.0, 0.2, 0.5, 0.7, NAN, 2.0]).to(dev)
    want = q.sample(x, torch.nan_to_num(u, nan=0.0).clamp(0, 1 - 2.0 ** -24))
    got = q.sample(x, u, **settings)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
