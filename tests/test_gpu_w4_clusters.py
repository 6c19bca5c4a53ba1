"""4-bit products where the device has no place for large clusters: the batches
that need them are multiplied by the other kernel instead of being refused."""

import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq, inputs
from tests.test_gpu_w4_linear import check, packed, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def restore():
    yield
    flexq.limit_clusters(0)


@pytest.mark.parametrize("most", [1, 2, 4])
@pytest.mark.parametrize("M, N, K, gs", [(1, 300, 4096, 128), (16, 500, 28672, 128), (9, 100, 28672, 64),
                                         (12, 3000, 8192, 32), (40, 300, 2048, 128), (300, 129, 4096, 256)])
def test_products_with_smaller_clusters(M, N, K, gs, most):
    wp, ws, w64 = packed(weights(N, K, N), gs)
    x = inputs.activations(M, K, seed=M)
    flexq.limit_clusters(most)
    y = flexq.linear4(x.cuda(), wp, ws, N, gs)
    check(y, x, w64, torch.float16, gs)
    assert flexq.device_status()[0] == flexq.FLEXQ_OK


def test_the_device_decides_without_a_limit():
    assert flexq.linear4_exact(16, 28672, 128)
    flexq.limit_clusters(4)
    assert not flexq.linear4_exact(16, 28672, 128)
