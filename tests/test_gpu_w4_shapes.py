"""4-bit products at the ends of the kernels' ranges: layers whose strips a
cluster takes in several rounds, for every group size and both numbers of
tokens that the streaming kernel multiplies at once, and long batches."""

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq, inputs
from tests.test_gpu_w4_linear import check, packed, weights
from tests.w4_util import dequantize, unpack4

pytestmark = pytest.mark.gpu


def rounds(M, N, K):
    """Rounds of a cluster of eight, by the shared memory that it has: 64 KB of
    buffers, the activations of its share of the columns, and 512 bytes per
    strip and eight tokens."""
    eights = 1 if M <= 8 else 2
    share = -(-(-(-K // 512)) // 8)
    room = 227 * 1024 - 256 - eights * 8192 - 65536 - M * (share * 1024 + 64)
    per_cluster = -(-(-(-N // 16)) // 15)         # at least, with 15 clusters or more
    return -(-per_cluster // (room // (512 * eights)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M, N, K, gs", [
    (16, 8192, 28672, 128), (16, 4500, 32768, 32), (16, 4500, 32768, 64), (15, 13000, 32768, 256),
    (8, 2000, 77824, 32), (8, 2000, 77824, 64), (8, 2000, 77824, 128), (8, 4001, 77824, 256)])
def test_layers_in_several_rounds(M, N, K, gs, dtype):
    assert flexq.linear4_exact(M, K, gs) and rounds(M, N, K) > 1
    strips, row_bytes = -(-N // 16), -(-K // 128) * 1024
    rng = np.random.default_rng(N + gs)
    b = rng.integers(0, 256, strips * row_bytes, dtype=np.uint8)
    s = (rng.random((N, K // gs)) * 0.02 + 0.001).astype(np.float16)
    x = inputs.activations(M, K, seed=gs).to(dtype)
    y = flexq.linear4(x.cuda(), torch.from_numpy(b).cuda(), torch.from_numpy(s).cuda(), N, gs).cpu()
    # every round has some of these strips: each fifth, and the last ones
    step = max(5, strips // 40)
    for strip in sorted({*range(0, strips, step), strips - 2, strips - 1}):
        r0, r1 = 16 * strip, min(N, 16 * strip + 16)
        q = unpack4(b[strip * row_bytes:(strip + 1) * row_bytes], r1 - r0, K)
        check(y[:, r0:r1], x, dequantize(q, s[r0:r1]), dtype, gs)
    assert flexq.device_status()[0] == flexq.FLEXQ_OK


@pytest.mark.parametrize("M, N, K, gs", [(2049, 300, 256, 64), (4100, 520, 512, 128), (20001, 40, 96, 32)])
def test_long_batches(M, N, K, gs):
    wp, ws, w64 = packed(weights(N, K, 31), gs)
    x = inputs.activations(M, K, seed=1)
    check(flexq.linear4(x.cuda(), wp, ws, N, gs), x, w64, torch.float16, gs)
