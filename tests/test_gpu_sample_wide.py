"""Sampling where a row keeps too many columns to be drawn from one by one: the chunks' sums
lead to the column.  Every combination of top-k, top-p and min-p, with min-p on either side of
the others' threshold."""
import numpy as np
import pytest
import torch

from qmm_testlib import require_gpu, values
from test_gpu_sample import check_row, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1500, 5000, 60000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_wide_cuts_match_float64(n, dtype):
    import bit_affine_quantized_qmv_amd as q
    dev = require_gpu()
    cases = [(k, p, m) for k in (0, 3 * n // 4, n // 2, 2 * n) for p in (1.0, 0.97, 0.6) for m in (0.0, 1e-4, 0.05, 0.6)]
    rows = len(cases)
    x = logits_of(rows, n, dtype, n, spread=1.5)
    k, p, m = (np.array(c, t) for c, t in zip(zip(*cases), (np.int32, np.float32, np.float32)))
    t = np.full(rows, 1.3, np.float32)
    u = np.random.default_rng(n).random(rows).astype(np.float32)
    u[::7] = 1.0                                            # the last column of the kept ones
    idx, prob = q.sample(x.to(dev), torch.from_numpy(u).to(dev), torch.from_numpy(t).to(dev),
                         torch.from_numpy(k).to(dev), torch.from_numpy(p).to(dev), torch.from_numpy(m).to(dev))
    torch.cuda.synchronize()
    l = values(x)
    for r in range(rows):
        check_row(int(idx[r]), float(prob[r]), l[r], u[r], float(t[r]), int(k[r]), float(p[r]), float(m[r]))
