"""Weights at the end of FP16's range: the quantizer's largest scale, 9360, is
that of a group whose maximum is near 65504, and 7 * 9360 lies between FP16's
largest value and infinity.  Every batch size and type multiplies such a group
with finite weights."""

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq
from tests.test_gpu_w4_linear import check, packed, weights
from tests.w4_util import pack4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gs", [32, 64, 256])
@pytest.mark.parametrize("M", [1, 16, 17, 40, 100, 300])
def test_groups_at_the_largest_weight(M, gs, dtype):
    N, K = 300, 768
    w = weights(N, K, 21)
    w[3, :gs] = 65504
    w[4, gs:2 * gs] = -65504
    w[5, -gs:] = torch.linspace(-65504, 65504, gs).half()
    w[200, :gs] = torch.linspace(-65488, 100, gs).half()
    wp, ws, w64 = packed(w, gs)
    assert float(ws.max()) == 9360.0
    # activations of 2^-12 and both signs: results stay below 65504
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M))
    x = (x * 2.0 ** -12).to(dtype)
    y = flexq.linear4(x.cuda(), wp, ws, N, gs)
    assert torch.isfinite(y).all()
    # 7 * 9360 becomes 65504, 16 / 65520 off: within half a step of FP16
    check(y, x, w64, dtype, gs)


@pytest.mark.parametrize("M", [20, 200])
def test_other_scales_round_as_before(M):
    # the largest scale changes the weights that would be infinite and no others
    N, K, gs = 16, 256, 128
    q = np.tile(np.arange(-7, 8).astype(np.int8), N * K // 15 + 1)[:N * K].reshape(N, K)
    s = np.array([9360, 9352, 9344, 1, 2.0 ** -24, 0.01, 3, 100] * 4, np.float16).reshape(N, 2)
    x = torch.zeros(M, K, dtype=torch.float16)
    for m in range(min(M, K)):
        x[m, m] = 0.5                          # picks out one column's weights
    y = flexq.linear4(x.cuda(), torch.from_numpy(pack4(q).copy()).cuda(), torch.from_numpy(s).cuda(), N, gs)
    with np.errstate(over="ignore"):
        w = (q.astype(np.float64) * np.repeat(s.astype(np.float64), gs, axis=1)).astype(np.float16)
    w = np.clip(w.astype(np.float64), -65504, 65504)
    want = (0.5 * w).astype(np.float16)[:, :min(M, K)].T
    assert np.array_equal(y.cpu().numpy()[:min(M, K)], want)
