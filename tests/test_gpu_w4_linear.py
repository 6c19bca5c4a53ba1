"""4-bit weights on the GPU: the quantizer bit for bit against its plain form,
and the linear layers against 64-bit sums.

Tolerance of an output: half a rounding step of its type, and the FP32 sums'
error: a product passes through at most 16 additions inside a tensor-core step
of 16 columns, 8 steps per tile of 128 columns, one addition per tile of its
warp, 8 warps and 8 cluster ranks, each off by at most 2^-23 (a truncation) of
the sum of magnitudes.  FP16 results below the normal range are off by half
of 2^-24."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq, inputs
from tests.w4_util import dequantize, half_step, pack4, quantize4, to64

pytestmark = pytest.mark.gpu


def weights(N, K, seed):
    return inputs.weights(N, K, seed=seed)


def packed(w, gs):
    wp, ws = flexq.quantize_weight4(w.cuda(), gs)
    q, s = quantize4(w.numpy(), gs)
    return wp, ws, dequantize(q, s)


def check(y, x, w64, dtype, gs, tokens=None):
    x64, tokens = to64(x), x.shape[0] if tokens is None else tokens
    ref, mags = x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
    tiles = -(-x64.shape[1] // 128)
    tol = (half_step(dtype) * np.abs(ref) + (48 + tiles) * 2.0 ** -23 * mags + 2.0 ** -25)
    if not flexq.linear4_exact(tokens, x64.shape[1], gs):
        tol += half_step(dtype) * mags + 2.0 ** -25 * np.abs(x64).sum(1, keepdims=True)
    bad = np.abs(to64(y) - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(to64(y) - ref).max()}"


def _edge_weights():
    w = weights(16, 256, 5)
    w[0, :32] = 0                                       # a group of zeros
    w[1, :32] = 2.0 ** -24                              # its scale underflows to zero
    w[2, :32] = torch.linspace(-6e-7, 6e-7, 32)         # a subnormal scale
    w[3, :32] = 7 * torch.tensor([0.5, -0.5, 1.5, 1, 2.5 / 7, -3.5 / 7, 7, -7] * 4)   # ties
    w[4, 32:64] = 65504                                 # the largest scale
    return w


@pytest.mark.parametrize("N, K, gs", [(1, 32, 32), (16, 128, 128), (19, 288, 32), (33, 320, 64),
                                      (100, 512, 256), (257, 1024, 128)])
def test_quantizer_matches_its_plain_form(N, K, gs):
    w = weights(N, K, N + K)
    wp, ws = flexq.quantize_weight4(w.cuda(), gs)
    q, s = quantize4(w.numpy(), gs)
    assert np.array_equal(ws.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert np.array_equal(wp.cpu().numpy(), pack4(q))


def test_quantizer_edge_values():
    w = _edge_weights()
    wp, ws = flexq.quantize_weight4(w.cuda(), 32)
    q, s = quantize4(w.numpy(), 32)
    assert np.array_equal(ws.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert np.array_equal(wp.cpu().numpy(), pack4(q))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M, N, K, gs", [
    (1, 1, 32, 32), (1, 100, 160, 32), (2, 16, 128, 128), (3, 257, 288, 32), (5, 33, 320, 64),
    (7, 48, 192, 64), (8, 1000, 1024, 128), (9, 65, 512, 256), (16, 31, 4096, 128),
    (17, 129, 768, 256), (31, 40, 2080, 32), (33, 77, 1088, 64), (64, 130, 1024, 256),
    (12, 700, 7168, 32), (16, 2400, 32768, 32), (16, 1500, 17408, 128), (32, 2500, 8192, 64), (24, 400, 28672, 256),
    (70, 129, 640, 128), (130, 300, 1024, 64), (300, 515, 2304, 256), (1, 4096, 4096, 128)])
def test_linear_against_64_bits(M, N, K, gs, dtype):
    wp, ws, w64 = packed(weights(N, K, 3 * N + K), gs)
    x = inputs.activations(M, K, seed=M).to(dtype)
    y = flexq.linear4(x.cuda(), wp, ws, N, gs)
    assert y.dtype == dtype and y.shape == (M, N)
    check(y, x, w64, dtype, gs)


@pytest.mark.parametrize("M", [1, 12, 200])
def test_every_code_is_multiplied_exactly(M):
    # codes -8 .. 7 in every place of a word, scales that are powers of two and
    # activations of -2 .. 2: every sum is an integer multiple that FP32 holds
    N, K, gs = 64, 512, 64
    rng = np.random.default_rng(M)
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    s = (2.0 ** rng.integers(-3, 1, (N, K // gs))).astype(np.float16)
    x = torch.from_numpy(rng.integers(-2, 3, (M, K)).astype(np.float16))
    y = flexq.linear4(x.cuda(), torch.from_numpy(pack4(q).copy()).cuda(),
                      torch.from_numpy(s).cuda(), N, gs)
    ref = (x.double().numpy() @ dequantize(q, s).T).astype(np.float16)
    assert np.array_equal(y.cpu().numpy(), ref)


@pytest.mark.parametrize("M", [1, 6, 40, 150])
def test_grouped_layers(M):
    K, gs = 1024, 128
    Ns = [500, 16, 77, 1]
    layers = [packed(weights(n, K, n), gs) for n in Ns]
    x = inputs.activations(M, K, seed=2)
    ys = flexq.linear4_group(x.cuda(), [(wp, ws, n) for (wp, ws, _), n in zip(layers, Ns)], gs)
    for y, (_, _, w64) in zip(ys, layers):
        check(y, x, w64, torch.float16, gs)


@pytest.mark.parametrize("M", [3, 20, 140])
def test_rows_of_wider_matrices(M):
    # x and out are column slices; what lies beside them is neither read into
    # the sums nor written
    N, K, gs = 50, 288, 32
    wp, ws, w64 = packed(weights(N, K, 9), gs)
    wide = torch.full((M, K + 64), float("nan"), dtype=torch.float16)
    x = inputs.activations(M, K, seed=4)
    wide[:, 32:32 + K] = x
    out = torch.full((M, N + 9), 7.0, dtype=torch.float16, device="cuda")
    y = flexq.linear4(wide.cuda()[:, 32:32 + K], wp, ws, N, gs, out=out[:, 4:4 + N])
    check(y, x, w64, torch.float16, gs)
    assert (out[:, :4] == 7).all() and (out[:, 4 + N:] == 7).all()


@pytest.mark.parametrize("M", [9, 100])
def test_special_values_stay_in_their_token(M):
    N, K, gs = 40, 512, 128
    wp, ws, w64 = packed(weights(N, K, 11), gs)
    x = inputs.activations(M, K, seed=6)
    bad = x.clone()
    bad[2, 5], bad[4, 100] = float("nan"), float("inf")
    y = flexq.linear4(bad.cuda(), wp, ws, N, gs)
    assert torch.isnan(y[2]).all()
    assert not torch.isfinite(y[4]).all()
    keep = [m for m in range(M) if m not in (2, 4)]
    check(y[keep], x[keep], w64, torch.float16, gs, tokens=M)


def test_no_tokens():
    wp, ws, _ = packed(weights(16, 128, 1), 128)
    y = flexq.linear4(torch.empty(0, 128, dtype=torch.float16, device="cuda"), wp, ws, 16, 128)
    assert y.shape == (0, 16)


@pytest.mark.parametrize("M", [1, 24, 160])
def test_repeats_captured_and_on_another_stream(M):
    N, K, gs = 300, 2048, 128
    wp, ws, w64 = packed(weights(N, K, 8), gs)
    x = inputs.activations(M, K, seed=1).cuda()
    first = flexq.linear4(x, wp, ws, N, gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = flexq.linear4(x, wp, ws, N, gs)
        out = torch.empty_like(first)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        flexq.linear4(x, wp, ws, N, gs, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, out)
    x2 = inputs.activations(M, K, seed=77)
    x.copy_(x2)
    graph.replay()
    check(out, x2, w64, torch.float16, gs)


def test_calls_on_two_streams_at_once():
    N, K, gs = 3000, 4096, 128
    wp, ws, _ = packed(weights(N, K, 8), gs)
    xs = [inputs.activations(m, K, seed=m).cuda() for m in (1, 12, 40, 300)]
    want = [flexq.linear4(x, wp, ws, N, gs) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        # the streams go through the batches in opposite directions
        for turn, stream in ((i, streams[0]), (3 - i, streams[1])):
            with torch.cuda.stream(stream):
                got.append((turn % 4, flexq.linear4(xs[turn % 4], wp, ws, N, gs)))
    torch.cuda.synchronize()
    for m, y in got:
        assert torch.equal(y, want[m])
    assert flexq.device_status()[0] == flexq.FLEXQ_OK


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_a_wait_that_runs_out_is_reported(M):
    N, K, gs = 300, 2048, 128
    wp, ws, w64 = packed(weights(N, K, 8), gs)
    x = inputs.activations(M, K, seed=1)
    assert flexq.device_status()[0] == flexq.FLEXQ_OK
    flexq.set_wait_limit_ns(50_000_000)          # 50 ms
    try:
        flexq.inject_stall(True)
        flexq.linear4(x.cuda(), wp, ws, N, gs)
        status, msg = flexq.device_status()
        assert status == flexq.FLEXQ_ERR_DEVICE_TIMEOUT, msg
        assert flexq.device_status()[0] == flexq.FLEXQ_OK     # cleared
    finally:
        flexq.inject_stall(False)
        flexq.set_wait_limit_ns(2_000_000_000)
    check(flexq.linear4(x.cuda(), wp, ws, N, gs), x, w64, torch.float16, gs)
    assert flexq.device_status()[0] == flexq.FLEXQ_OK


FIRST_CALLS = """
import torch
from bit_group_quantized_flexq_b200 import flexq
torch.manual_seed(0)
w = torch.randn(400, 1024, device="cuda").half()
wp, ws = flexq.quantize_weight4(w, 128)
ids = torch.randint(-1, 400, (700,), device="cuda")
xs = [torch.randn(m, 1024, device="cuda").half() for m in (1, 12, 40, 300)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ys = [flexq.linear4(x, wp, ws, 400, 128) for x in xs]
    e = flexq.embedding(ids, wp, ws, 400, 128)
    rows, scales = flexq.embedding_backward(e, ids, wp, 400, 128, table_dtype=torch.float16)
graph.replay()
torch.cuda.synchronize()
for x, y in zip(xs, ys):
    assert torch.equal(y, flexq.linear4(x, wp, ws, 400, 128)), x.shape
assert torch.equal(e, flexq.embedding(ids, wp, ws, 400, 128))
again = flexq.embedding_backward(e, ids, wp, 400, 128, table_dtype=torch.float16)
assert torch.equal(rows, again[0]) and torch.equal(scales, again[1])
print("same")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True,
                       timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_scales_written_just_before_are_the_ones_used():
    # a step of scale tuning: the scales change in place between two products
    N, K, gs = 700, 4096, 128
    wp, ws, _ = packed(weights(N, K, 3), gs)
    for M in (1, 12, 40, 300):
        x = inputs.activations(M, K, seed=M).cuda()
        s = ws.clone()
        y = flexq.linear4(x, wp, s, N, gs)
        for _ in range(4):
            s.mul_(0.5)
            half = flexq.linear4(x, wp, s, N, gs)
            # halving is exact down to subnormal results
            assert torch.allclose(half.float() * 2, y.float(), rtol=2.0 ** -9, atol=2.0 ** -22)
            y = half


def test_codes_written_just_before_are_the_ones_used():
    # weights exchanged in place between two products, eagerly and replayed
    N, K, gs = 700, 4096, 128
    wa, ws, _ = packed(weights(N, K, 3), gs)
    wb, _, _ = packed(weights(N, K, 4), gs)
    for M in (1, 12, 40, 300):
        x = inputs.activations(M, K, seed=M).cuda()
        want = [flexq.linear4(x, w, ws, N, gs) for w in (wa, wb)]
        assert not torch.equal(*want)
        w = wa.clone()
        graph = torch.cuda.CUDAGraph()
        got = []
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for i in range(8):
                w.copy_((wb, wa)[i % 2])
                got.append(flexq.linear4(x, w, ws, N, gs))
        graph.replay()
        for i, y in enumerate(got):
            assert torch.equal(y, want[(i + 1) % 2]), (M, i)
        for i in range(8):
            w.copy_((wb, wa)[i % 2])
            assert torch.equal(flexq.linear4(x, w, ws, N, gs), want[(i + 1) % 2]), (M, i)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [2, 16, 40, 300])
def test_a_token_that_is_not_finite_stays_alone(M, dtype):
    N, K, gs = 300, 1024, 64
    wp, ws, w64 = packed(weights(N, K, 8), gs)
    x = inputs.activations(M, K, seed=2).to(dtype)
    want = flexq.linear4(x.cuda(), wp, ws, N, gs)
    for m, value in ((0, float("nan")), (M - 1, float("inf"))):
        bad = x.clone()
        bad[m, 700] = value
        y = flexq.linear4(bad.cuda(), wp, ws, N, gs)
        assert not torch.isfinite(y[m]).any()
        rest = [i for i in range(M) if i != m]
        assert torch.equal(y[rest], want[rest])


def test_refusals_on_the_gpu():
    wp, ws, _ = packed(weights(16, 256, 1), 128)
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        flexq.linear4(x, wp, ws, 17 + 16, 128)
    with pytest.raises(ValueError, match="shape"):
        flexq.linear4(x, wp, ws.t().contiguous(), 16, 128)
    with pytest.raises(ValueError, match="contiguous rows"):
        flexq.linear4(torch.zeros(256, 4, dtype=torch.float16, device="cuda").t(), wp, ws, 16, 128)
    with pytest.raises(flexq.FlexQError, match="multiple of 8"):
        flexq.linear4(torch.zeros(4, 260, dtype=torch.float16, device="cuda")[:, :256], wp, ws, 16, 128)
    with pytest.raises(flexq.FlexQError, match="16-byte aligned"):
        flexq.linear4(torch.zeros(4, 264, dtype=torch.float16, device="cuda")[:, 4:260], wp, ws, 16, 128)
    with pytest.raises(flexq.FlexQError, match="below"):
        flexq.linear4(x[:1].expand(4, 256), wp, ws, 16, 128)
    with pytest.raises(ValueError, match="out must be"):
        flexq.linear4(x, wp, ws, 16, 128, out=torch.zeros(4, 16, device="cuda"))
    with pytest.raises(flexq.FlexQError, match="unsupported"):
        flexq.linear4(x[:, :160], wp, ws, 16, 128)
    with pytest.raises(ValueError, match="layers"):
        flexq.linear4_group(x, [(wp, ws, 16)] * 5, 128)
