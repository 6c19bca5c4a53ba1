"""Which batches the streaming kernel takes, by the clusters that are there."""

import pytest

from bit_group_quantized_flexq_b200 import build as flexq_build
from bit_group_quantized_flexq_b200 import flexq


@pytest.fixture(scope="module", autouse=True)
def built():
    flexq_build.build()
    yield
    flexq.limit_clusters(0)


def test_batches_that_need_a_cluster_are_not_exact_without_one():
    # activations of 16 tokens x 28672 columns are 917 KB: eight shares of them
    # fit the SMs' shared memory, four and fewer do not
    for most, exact in [(0, True), (8, True), (4, False), (1, False), (0, True)]:
        flexq.limit_clusters(most)
        assert flexq.linear4_exact(16, 28672, 128) is exact
        assert flexq.linear4_exact(1, 4096, 128)


def test_invalid_limits_are_refused():
    for most in (-1, 9):
        with pytest.raises(flexq.FlexQError, match="0..8"):
            flexq.limit_clusters(most)
