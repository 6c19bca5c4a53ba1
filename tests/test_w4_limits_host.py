"""Batches next to the largest int: the kernels number a tile's tokens past the
last one, so the last 127 counts are refused before anything is computed."""

import ctypes

import pytest

from bit_group_quantized_flexq_b200 import build as flexq_build
from bit_group_quantized_flexq_b200 import flexq

FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    flexq_build.build()
    return flexq.lib()


@pytest.mark.parametrize("M", [INT_MAX, INT_MAX - 126])
def test_token_counts_that_a_tile_would_pass(L, M):
    rc = L.flexq_linear_w4(M, 1, 32, 32, 0, FAKE, 32, FAKE, FAKE, FAKE, 1, None)
    assert rc == flexq.FLEXQ_ERR_UNSUPPORTED
    assert b"too large" in L.flexq_last_error_message()
    layer = (flexq.Layer4 * 1)(flexq.Layer4(1, 1 << 20, 1 << 20, 1 << 20, 1))
    assert L.flexq_linear_w4_group(M, 32, 32, 0, FAKE, 32, 1, layer, None) == flexq.FLEXQ_ERR_UNSUPPORTED
