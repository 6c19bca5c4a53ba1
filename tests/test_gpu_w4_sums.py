"""Batches that multiply the codes themselves, where the terms of a sum differ
much in size: an activation on a zero code costs the other terms nothing, and
no finite activation overflows a group's sum.

The tolerance is the one that a direct FP32 sum of x * q * s keeps, in units of
the sum of |x q s| (derived in test_gpu_w4_linear)."""

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq
from tests.test_gpu_w4_linear import check
from tests.w4_util import dequantize, half_step, pack4, to64

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]


def layer(q, s):
    """(packed codes, scales, 64-bit weights) of codes [N, K] and scales [N, G]."""
    return (torch.from_numpy(pack4(q).copy()).cuda(), torch.from_numpy(s).cuda(), dequantize(q, s))


def codes(N, K, gs, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(-7, 8, (N, K)).astype(np.int8)
    return q, (rng.random((N, K // gs)) * 0.02 + 0.001).astype(np.float16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gs", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 5, 16])
def test_a_large_channel_on_zero_codes_costs_nothing(M, gs, dtype):
    N, K = 100, 1024
    q, s = codes(N, K, gs, gs)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M))
    for c in (0, 200, 517, 1023):
        q[:, c] = 0
        x[:, c] = 30000.0 if c % 2 else -30000.0
    x = x.to(dtype)
    wp, ws, w64 = layer(q, s)
    assert flexq.linear4_exact(M, K, gs)
    check(flexq.linear4(x.cuda(), wp, ws, N, gs), x, w64, dtype, gs)
    # the same with the channel at zero: the same terms in the same order
    x0 = x.clone()
    x0[:, [0, 200, 517, 1023]] = 0
    assert torch.equal(flexq.linear4(x0.cuda(), wp, ws, N, gs), flexq.linear4(x.cuda(), wp, ws, N, gs))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 9])
def test_groups_of_one_code(M, dtype):
    # one code per group, and small activations there: 1/4096 of the others
    N, K, gs = 48, 2048, 128
    rng = np.random.default_rng(M)
    q = np.zeros((N, K), np.int8)
    at = rng.integers(0, gs, (N, K // gs)) + np.arange(K // gs) * gs
    at = at // 16 * 16 + 3                       # shared by few columns, so that those can be small
    np.put_along_axis(q, at, 7, axis=1)
    s = (rng.random((N, K // gs)) * 0.02 + 0.001).astype(np.float16)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(0))
    x[:, 3::16] /= 4096
    x = x.to(dtype)
    wp, ws, w64 = layer(q, s)
    y = flexq.linear4(x.cuda(), wp, ws, N, gs)
    check(y, x, w64, dtype, gs)
    # the bound that check leaves at results this small, without its constant
    ref, mags = to64(x) @ w64.T, np.abs(to64(x)) @ np.abs(w64).T
    err = np.abs(to64(y) - ref)
    assert (err <= half_step(dtype) * np.abs(ref) + 64 * 2.0 ** -23 * mags + 2.0 ** -25).all()


@pytest.mark.parametrize("gs", [32, 256])
@pytest.mark.parametrize("M", [1, 16])
def test_no_finite_bfloat16_overflows_a_sum(M, gs):
    # the largest activations: a group's sum of x q reaches gs * 7 * 3.4e38,
    # and the scales bring the result back
    N, K = 33, 512
    q = np.full((N, K), 7, np.int8)
    q[1] = -8
    q[2, ::2] = -7
    s = np.full((N, K // gs), 2.0 ** -20, np.float16)
    big = torch.finfo(torch.bfloat16).max
    x = torch.full((M, K), big).to(torch.bfloat16)
    if M > 1:
        x[1] = -big
        x[2] = 2.0 ** 100
    wp, ws, w64 = layer(q, s)
    y = flexq.linear4(x.cuda(), wp, ws, N, gs)
    assert torch.isfinite(y).all()
    check(y, x, w64, torch.bfloat16, gs)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [1, 16])
def test_an_infinite_activation_follows_the_formula(M, dtype):
    N, K, gs = 64, 256, 64
    q, s = codes(N, K, gs, 3)
    q[:8, 70] = 0
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 70] = float("inf")
    wp, ws, w64 = layer(q, s)
    y = to64(flexq.linear4(x.cuda(), wp, ws, N, gs))[0]
    assert np.isnan(y[q[:, 70] == 0]).all()               # infinity times zero
    some = q[:, 70] != 0
    assert np.array_equal(y[some], np.where(q[some, 70] > 0, np.inf, -np.inf))
