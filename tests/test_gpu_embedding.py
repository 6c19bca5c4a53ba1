"""Lookup of packed tables and its gradient against their 64-bit forms.

Lookup: code times scale is exact in FP32, the factor rounds once there
(2^-24) and the result once to its type.  Gradient: the n tokens of a row are
added in FP32 (n additions and the factor, 2^-24 each, of the sum of
magnitudes); the scales' gradient adds a group of gs products of those."""

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq, inputs
from oracle import flexq_oracle as orc
from tests.w4_util import (dequantize, embedding64, embedding_backward64, half_step, quantize4,
                           to64)

pytestmark = pytest.mark.gpu


def table(V, K, gs, bits, seed=0):
    """(packed, scales, codes, FP64 scales [V, G]) of a table."""
    w = inputs.weights(V, K, seed=inputs.layer_seed("table", V, K, seed))
    if bits == 4:
        q, s = quantize4(w.numpy(), gs)
        return flexq.quantize_weight4(w.cuda(), gs) + (q, s)
    q, s = orc.quantize_weight(w.numpy(), gs)
    return flexq.quantize_weight(w.cuda(), gs) + (np.asarray(q), np.asarray(s).reshape(V, -1))


SHAPES = [(100, 512, 128, 4), (1, 32, 32, 4), (33, 160, 32, 4), (1000, 2304, 256, 4),
          (70, 4160, 64, 4), (128, 256, 32, 6), (256, 512, 128, 6), (384, 2304, 256, 6)]


def test_oracle_scales_are_by_row():
    q, s = orc.quantize_weight(inputs.weights(128, 256, seed=1).numpy(), 64)
    assert np.asarray(s).shape == (128, 4)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("V, K, gs, bits", SHAPES)
def test_lookup(V, K, gs, bits, id_type, dtype):
    wp, ws, q, s = table(V, K, gs, bits)
    w64 = dequantize(q, s)
    for shape, scale in [((), 1.0), ((3,), 1.0), ((2, 67), K ** 0.5)]:
        ids = torch.randint(-1, V + 1, shape, generator=torch.Generator().manual_seed(K), dtype=id_type)
        y = flexq.embedding(ids.cuda(), wp, ws, V, gs, scale=scale, weight_bits=bits, dtype=dtype)
        assert y.shape == (*shape, K) and y.dtype == dtype
        ref = embedding64(ids, w64, scale).reshape(y.shape)
        tol = (half_step(dtype) + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25
        assert (np.abs(to64(y) - ref) <= tol).all()


def test_lookup_reads_every_row_and_column():
    for V, K, gs, bits in [(130, 288, 32, 4), (256, 512, 64, 6)]:
        wp, ws, q, s = table(V, K, gs, bits)
        ids = torch.arange(V, dtype=torch.int32).cuda()
        y = flexq.embedding(ids, wp, ws, V, gs, weight_bits=bits)
        ref = (q.astype(np.float32) * np.repeat(s.astype(np.float32), gs, axis=1)).astype(np.float16)
        assert np.array_equal(y.cpu().numpy(), ref)


def test_lookup_extremes():
    V, K, gs = 20, 256, 64
    wp, ws, q, s = table(V, K, gs, 4)
    out = torch.full((3, K), 5.0, dtype=torch.float16, device="cuda")
    ids = torch.tensor([2 ** 40, -2 ** 40, 2 ** 32 + 3], device="cuda")   # padding, not row 3
    assert (flexq.embedding(ids, wp, ws, V, gs, out=out) == 0).all()
    assert flexq.embedding(ids[:0], wp, ws, V, gs).shape == (0, K)
    y = flexq.embedding(torch.tensor([1], device="cuda"), wp, ws, V, gs, scale=1e9)
    big = q[1] * np.repeat(s[1].astype(np.float64), gs)[None] * 1e9
    assert np.array_equal(np.isinf(to64(y)), np.abs(big) > 65520)


def _ids(kind, T, V, seed):
    rng = np.random.default_rng(seed)
    if kind == "same":
        return np.full(T, V // 2)
    if kind == "padding":
        return np.full(T, -1)
    if kind == "distinct":
        return rng.permutation(max(T, V))[:T] % V
    if kind == "heavy":                           # one row holds most tokens, some are padding
        ids = rng.integers(-1, V + 1, T)
        ids[rng.random(T) < 0.7] = V - 1
        return ids
    return rng.integers(0, V, T)


def check_backward(table_grad, scales_grad, dy, ids, q, gs, bits, scale, table_dtype):
    dy64 = to64(dy)
    V = q.shape[0]
    D, ds = embedding_backward64(dy64, ids, q, gs, scale)
    mags, _ = embedding_backward64(np.abs(dy64), ids, q, gs, abs(scale))
    count = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None]
    tol32 = (count + 2) * 2.0 ** -24 * mags
    if table_dtype is not None:
        tol = tol32 + half_step(table_dtype) * np.abs(D)
        if table_dtype != torch.float32:
            tol += 2.0 ** -25
        assert (np.abs(to64(table_grad) - D) <= tol).all()
        assert (to64(table_grad)[count[:, 0] == 0] == 0).all()
    else:
        assert table_grad is None
    if scales_grad is not None:
        got = to64(scales_grad) if bits == 4 else to64(scales_grad).T
        per = (np.abs(q) * (tol32 + (gs + 1) * 2.0 ** -24 * mags)).reshape(V, -1, gs).sum(-1)
        assert got.shape == ds.shape
        assert (np.abs(got - ds) <= per).all()


@pytest.mark.parametrize("V, K, gs, bits, T, kind, dtype, table_dtype", [
    (100, 512, 128, 4, 1, "any", torch.float16, torch.float16),
    (100, 512, 128, 4, 2, "same", torch.bfloat16, torch.float32),
    (33, 160, 32, 4, 37, "any", torch.float16, torch.float32),
    (1, 32, 32, 4, 70, "same", torch.float16, torch.float16),
    (3, 4160, 64, 4, 129, "any", torch.bfloat16, torch.bfloat16),
    (3, 4160, 64, 4, 128, "any", torch.float16, torch.float32),
    (2000, 160, 32, 4, 100, "heavy", torch.bfloat16, torch.bfloat16),
    (500, 96, 32, 4, 256, "heavy", torch.bfloat16, torch.float32),
    (500, 96, 32, 4, 257, "heavy", torch.float16, torch.float16),
    (128, 512, 64, 6, 700, "same", torch.float16, torch.float16),
    (300, 64, 64, 4, 40000, "heavy", torch.float16, torch.float32),
    (20001, 1024, 128, 4, 700, "heavy", torch.float16, torch.float32),    # 82 MB of rows
    (9088, 4096, 256, 6, 3000, "any", torch.bfloat16, torch.bfloat16),
    (128, 512, 64, 6, 128, "distinct", torch.float16, torch.float16),
    (384, 256, 256, 6, 77, "padding", torch.bfloat16, torch.float32),
    (1000, 256, 256, 4, 1024, "distinct", torch.float16, torch.float16),
    (1000, 2304, 256, 4, 1025, "heavy", torch.bfloat16, torch.float32),
    (300, 96, 32, 4, 5000, "same", torch.float16, torch.float16),
    (70000, 64, 64, 4, 4097, "heavy", torch.float16, None),
    (128, 256, 32, 6, 60, "heavy", torch.float16, torch.float16),
    (256, 2304, 256, 6, 2000, "any", torch.bfloat16, torch.bfloat16),
    (384, 512, 128, 6, 9000, "heavy", torch.float16, torch.float32),
    (50, 128, 128, 4, 33, "padding", torch.float16, torch.float16),
])
def test_gradient(V, K, gs, bits, T, kind, dtype, table_dtype):
    wp, ws, q, s = table(V, K, gs, bits)
    ids = _ids(kind, T, V, T)
    dy = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(dtype)
    dev = torch.from_numpy(ids).to(torch.int32 if T % 2 else torch.int64).cuda()
    args = (dy.cuda(), dev, wp, V, gs)
    kw = dict(scale=1.7, weight_bits=bits, table_dtype=table_dtype)
    rows, scales = flexq.embedding_backward(*args, **kw)
    check_backward(rows, scales, dy, ids, q, gs, bits, float(np.float32(1.7)), table_dtype)
    again = flexq.embedding_backward(*args, **kw)
    assert torch.equal(scales, again[1])
    if rows is not None:
        assert torch.equal(rows, again[0])
        alone, none = flexq.embedding_backward(*args, **kw, with_scales=False)
        assert none is None and torch.equal(rows, alone)


def test_padding_tokens_give_nothing_even_where_not_finite():
    V, K, gs = 40, 256, 64
    wp, ws, q, s = table(V, K, gs, 4)
    ids = np.array([3, -1, 3, V, 7])
    dy = torch.randn(5, K, generator=torch.Generator().manual_seed(0)).half()
    bad = dy.clone()
    bad[1], bad[3] = float("nan"), float("inf")
    rows, scales = flexq.embedding_backward(bad.cuda(), torch.from_numpy(ids).cuda(), wp, V, gs,
                                            table_dtype=torch.float32)
    check_backward(rows, scales, dy, ids, q, gs, 4, 1.0, torch.float32)


@pytest.mark.parametrize("bits", [4, 6])
def test_no_tokens_write_zeros(bits):
    V, K, gs = (41, 160, 32) if bits == 4 else (128, 256, 32)
    wp, ws, q, s = table(V, K, gs, bits)
    shape = (V, K // gs) if bits == 4 else (K // gs, V)
    out = (torch.full((V, K), 3.0, device="cuda"), torch.full(shape, 3.0, device="cuda"))
    rows, scales = flexq.embedding_backward(torch.empty(0, K, dtype=torch.float16, device="cuda"),
                                            torch.empty(0, dtype=torch.int64, device="cuda"), wp, V,
                                            gs, weight_bits=bits, table_dtype=torch.float32, out=out)
    assert rows is out[0] and scales is out[1]
    assert (rows == 0).all() and (scales == 0).all()


def test_scale_gradient_against_differences():
    # the lookup is linear in a scale: moving one by h moves the loss sum(dy *
    # y) by h * ds, up to the rounding of the looked-up FP16 values (half a
    # step each, twice)
    V, K, gs = 10, 128, 32
    wp, ws, q, s = table(V, K, gs, 4)
    ids = torch.tensor([4, 2, 4, 4, -1, 9]).cuda()
    dy = torch.randn(6, K, generator=torch.Generator().manual_seed(3)).half().cuda()
    _, scales = flexq.embedding_backward(dy, ids, wp, V, gs, scale=2.0)

    def values(w):
        return flexq.embedding(ids, wp, w, V, gs, scale=2.0)

    for v, g in [(4, 0), (4, 3), (2, 1), (0, 2)]:
        up, down = ws.clone(), ws.clone()
        h = float(s[v, g]) / 4
        up[v, g] += h
        down[v, g] -= h
        step = float(up[v, g].double() - down[v, g].double())
        yu, yd = values(up), values(down)
        diff = float((dy.double() * (yu.double() - yd.double())).sum()) / step
        changed = (ids == v)[:, None] & (torch.arange(K, device="cuda") // gs == g)
        err = (dy.double().abs() * (yu.double().abs() + yd.double().abs()) * changed).sum()
        assert abs(diff - float(scales[v, g])) <= float(err) * 2.0 ** -11 / step + 1e-5


@pytest.mark.parametrize("bits", [4, 6])
def test_lookup_of_more_tokens_than_a_launch_takes_at_once(bits):
    V, K, gs = 128, 256, 64
    wp, ws, q, s = table(V, K, gs, bits)
    ids = torch.randint(-1, V + 1, (100003,), generator=torch.Generator().manual_seed(5))
    y = flexq.embedding(ids.cuda(), wp, ws, V, gs, weight_bits=bits)
    rows = (q.astype(np.float32) * np.repeat(s.astype(np.float32), gs, axis=1)).astype(np.float16)
    rows = np.concatenate([rows, np.zeros((1, K), np.float16)])
    at = np.where((ids.numpy() >= 0) & (ids.numpy() < V), ids.numpy(), V)
    assert np.array_equal(y.cpu().numpy(), rows[at])


def test_captured_and_replayed_beside_another_stream():
    V, K, gs, T = 500, 1024, 128, 3000
    wp, ws, q, s = table(V, K, gs, 4)
    ids = torch.from_numpy(_ids("heavy", T, V, 1)).cuda()
    dy = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).half().cuda()
    want = flexq.embedding_backward(dy, ids, wp, V, gs, table_dtype=torch.float16)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y = flexq.embedding(ids, wp, ws, V, gs)
        rows, scales = flexq.embedding_backward(dy, ids, wp, V, gs, table_dtype=torch.float16)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):                         # the graph and eager calls run at the same time
        graph.replay()
        with torch.cuda.stream(other):
            beside = flexq.embedding_backward(dy, ids, wp, V, gs, table_dtype=torch.float16)
    torch.cuda.synchronize()
    for got in [(rows, scales), beside]:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ids.copy_(torch.from_numpy(_ids("any", T, V, 2)))
    graph.replay()
    torch.cuda.synchronize()
    check_backward(rows, scales, dy, ids.cpu().numpy(), q, gs, 4, 1.0, torch.float16)
    assert np.array_equal(to64(y), to64(flexq.embedding(ids, wp, ws, V, gs)))


def test_refusals_on_the_gpu():
    V, K, gs = 40, 256, 64
    wp, ws, q, s = table(V, K, gs, 4)
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    dy = torch.zeros(3, K, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="weight_bits"):
        flexq.embedding(ids, wp, ws, V, gs, weight_bits=5)
    with pytest.raises(flexq.FlexQError, match="unsupported"):
        flexq.embedding(ids, wp, ws, V, gs, weight_bits=6)
    with pytest.raises(ValueError, match="shape"):
        flexq.embedding(ids, wp, ws, V + 16, gs)
    with pytest.raises(ValueError, match="dtype"):
        flexq.embedding(ids, wp, ws, V, gs, dtype=torch.float32)
    with pytest.raises(ValueError, match="contiguous"):
        flexq.embedding(torch.zeros(6, dtype=torch.int64, device="cuda")[::2], wp, ws, V, gs)
    with pytest.raises(ValueError, match="shape"):
        flexq.embedding_backward(dy[:2], ids, wp, V, gs)
    with pytest.raises(ValueError, match="table_dtype"):
        flexq.embedding_backward(dy, ids, wp, V, gs, table_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="nothing to compute"):
        flexq.embedding_backward(dy, ids, wp, V, gs, with_scales=False)
    with pytest.raises(flexq.FlexQError, match="workspace"):
        many = torch.zeros(300, dtype=torch.int64, device="cuda")
        flexq.embedding_backward(torch.zeros(300, K, dtype=torch.float16, device="cuda"), many, wp, V, gs,
                                 workspace_buf=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        flexq.embedding_backward(dy[:, ::2][:, :128].expand(3, 128), ids, wp, V, gs)


@pytest.mark.parametrize("bits", [4, 6])
def test_tied_table_from_tokens_to_logits(bits):
    # the table looked up at the input and multiplied as the output head
    V, K, gs = 256, 512, 128
    wp, ws, q, s = table(V, K, gs, bits)
    ids = torch.tensor([[5, 17, -1], [255, 0, 5]]).cuda()
    x = flexq.embedding(ids, wp, ws, V, gs, scale=4.0, weight_bits=bits).flatten(0, 1)
    w64 = dequantize(q, s)
    if bits == 4:
        logits = flexq.linear4(x, wp, ws, V, gs)
        ref, mags = to64(x) @ w64.T, np.abs(to64(x)) @ np.abs(w64).T
        tol = half_step(torch.float16) * np.abs(ref) + (48 + 4) * 2.0 ** -23 * mags + 2.0 ** -25
        assert (np.abs(to64(logits) - ref) <= tol).all()
        dy = torch.randn(2, 3, K, generator=torch.Generator().manual_seed(0)).half()
        rows, scales = flexq.embedding_backward(dy.cuda(), ids, wp, V, gs, scale=4.0,
                                                table_dtype=torch.float16)
        check_backward(rows, scales, dy.reshape(6, K), ids.cpu().numpy().reshape(-1), q, gs, 4, 4.0,
                       torch.float16)
    else:
        logits = flexq.linear(x, wp, ws, V, gs, 8)
    assert (logits[2] == 0).all()                 # padding looks up zeros
    assert int(logits[0].argmax()) == int(logits[5].argmax()) == 5
