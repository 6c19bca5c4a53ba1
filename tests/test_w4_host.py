"""The 4-bit layers and packed tables without a GPU: sizes, refusals before
anything is enqueued, and the packed form as the header words it."""

import ctypes

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import build as flexq_build
from bit_group_quantized_flexq_b200 import flexq
from tests.w4_util import pack4, unpack4

FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)
NULL = ctypes.c_void_p(0)
INVALID, UNSUPPORTED, BAD_ALIGN = (flexq.FLEXQ_ERR_INVALID_ARG, flexq.FLEXQ_ERR_UNSUPPORTED,
                                   flexq.FLEXQ_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def L():
    flexq_build.build()
    return flexq.lib()


def test_packed_size(L):
    assert flexq.weight4_packed_bytes(4096, 4096, 128) == 4096 * 4096 // 2
    assert flexq.weight4_packed_bytes(1, 32, 32) == 1024             # one padded tile
    assert flexq.weight4_packed_bytes(17, 160, 32) == 2 * 2 * 1024
    for bad in [(0, 256, 32), (16, 0, 32), (16, 160, 64), (16, 256, 48), (-1, 256, 32)]:
        assert flexq.weight4_packed_bytes(*bad) == 0


def test_the_packed_form_by_plain_index_arithmetic():
    rng = np.random.default_rng(0)
    N, K = 19, 288
    q = rng.integers(-8, 8, (N, K)).astype(np.int8)
    b = pack4(q)
    assert b.size == 2 * 3 * 1024
    for n, k in [(0, 0), (0, 1), (3, 9), (15, 127), (16, 128), (18, 287), (7, 200)]:
        tile = (n // 16) * 3 + k // 128
        kk, r = k % 128, n % 16
        w, t, i = kk // 32, kk // 8 % 4, kk % 8
        nibble = [0, 4, 2, 6, 1, 5, 3, 7][i]
        byte = b[tile * 1024 + r * 64 + t * 16 + w * 4 + nibble // 2]
        assert (int(byte) >> (4 * (nibble % 2))) & 15 == q[n, k] + 8
    assert np.array_equal(unpack4(b, N, K), q)


def test_which_batches_multiply_the_codes_themselves(L):
    for M, K, gs in [(1, 32, 32), (1, 28672, 128), (8, 28672, 32), (16, 28672, 128), (16, 8192, 64)]:
        assert flexq.linear4_exact(M, K, gs)
    for M, K, gs in [(17, 256, 128), (16, 65536, 128), (2048, 4096, 64), (0, 256, 128),
                     (1, 200, 128), (1, 1 << 22, 128)]:
        assert not flexq.linear4_exact(M, K, gs)


def test_linear_refusals_before_any_launch(L):
    f = L.flexq_linear_w4
    ok = (4, 100, 256, 128, 0, FAKE, 256, FAKE, FAKE, FAKE, 100, NULL)

    def call(**kw):
        names = ["M", "N", "K", "gs", "dtype", "X", "ldx", "Wq", "Ws", "Y", "ldy", "stream"]
        return f(*[kw.get(n, v) for n, v in zip(names, ok)])

    assert call(M=-1) == INVALID
    assert call(N=0) == INVALID
    assert call(gs=48) == UNSUPPORTED
    assert call(K=200, ldx=200) == UNSUPPORTED
    assert call(dtype=2) == INVALID
    assert call(X=NULL) == INVALID and b"X" in L.flexq_last_error_message()
    assert call(X=MISALIGNED) == BAD_ALIGN
    assert call(ldx=128) == INVALID
    assert call(ldx=260) == BAD_ALIGN
    assert call(Wq=NULL) == INVALID
    assert call(Ws=MISALIGNED) == BAD_ALIGN
    assert call(Y=NULL) == INVALID
    assert call(ldy=99) == INVALID
    assert call(M=0, X=NULL, Y=NULL) == flexq.FLEXQ_OK
    g = L.flexq_linear_w4_group
    arr = (flexq.Layer4 * 1)(flexq.Layer4(100, 1 << 20, 1 << 20, 1 << 20, 100))
    assert g(4, 256, 128, 0, FAKE, 256, 0, arr, NULL) == INVALID
    assert g(4, 256, 128, 0, FAKE, 256, 5, arr, NULL) == INVALID
    assert g(4, 256, 128, 0, FAKE, 256, 1, None, NULL) == INVALID
    assert L.flexq_quantize_weight4(16, 200, 64, FAKE, FAKE, FAKE, NULL) == UNSUPPORTED
    assert L.flexq_quantize_weight4(16, 256, 64, FAKE, NULL, FAKE, NULL) == INVALID
    assert L.flexq_quantize_weight4(16, 256, 64, MISALIGNED, FAKE, FAKE, NULL) == BAD_ALIGN


def test_embedding_refusals_before_any_launch(L):
    f = L.flexq_embedding
    ok = dict(T=4, V=100, K=256, gs=128, bits=4, dtype=0, ids=FAKE, id_bytes=8, Wq=FAKE, Ws=FAKE,
              scale=1.0, out=FAKE, stream=NULL)

    def call(**kw):
        return f(*[kw.get(n, v) for n, v in ok.items()])

    assert call(bits=5) == INVALID
    assert call(bits=6) == UNSUPPORTED                 # 100 rows: the 6-bit form has 128-row tiles
    assert call(T=-1) == INVALID
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(dtype=2) == INVALID
    assert call(id_bytes=2) == INVALID
    assert call(V=0) == INVALID
    assert call(K=200) == UNSUPPORTED
    assert call(ids=NULL) == INVALID
    assert call(ids=ctypes.c_void_p((1 << 20) + 4)) == BAD_ALIGN
    assert call(Wq=NULL) == INVALID
    assert call(out=MISALIGNED) == BAD_ALIGN
    assert call(T=0, ids=NULL, out=NULL) == flexq.FLEXQ_OK


def test_embedding_backward_refusals_before_any_launch(L):
    f = L.flexq_embedding_backward
    need = flexq.embedding_backward_workspace_bytes(400, 100, 256)
    assert need > 0
    assert flexq.embedding_backward_workspace_bytes(0, 100, 256) == 0
    assert flexq.embedding_backward_workspace_bytes(256, 100, 256) == 0     # one launch, no scratch
    ok = dict(T=400, V=100, K=256, gs=128, bits=4, dtype=0, ids=FAKE, id_bytes=8, dY=FAKE, Wq=FAKE,
              scale=1.0, table_dtype=0, table=FAKE, scales=FAKE, ws=FAKE, ws_bytes=need,
              stream=NULL)

    def call(**kw):
        return f(*[kw.get(n, v) for n, v in ok.items()])

    assert call(table=NULL, scales=NULL) == INVALID
    assert call(table_dtype=1) == INVALID              # neither dY's type nor FP32
    assert call(table=MISALIGNED) == BAD_ALIGN
    assert call(scales=MISALIGNED) == BAD_ALIGN
    assert call(dY=NULL) == INVALID
    assert call(ids=NULL) == INVALID
    assert call(ws=NULL) == INVALID
    assert call(ws_bytes=need - 1) == INVALID
    assert call(Wq=NULL) == INVALID                    # the scales' gradient reads the codes
    assert call(bits=6) == UNSUPPORTED
    assert call(T=-5) == INVALID


def test_python_refusals():
    x = torch.zeros(2, 256, dtype=torch.float16)
    wp, ws = torch.zeros(16 * 128, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        flexq.linear4(x, wp, ws, 16, 128)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        flexq.linear4(x.float(), wp, ws, 16, 128)
    with pytest.raises(TypeError):
        flexq.linear4(None, wp, ws, 16, 128)
    with pytest.raises(ValueError, match="int32"):
        flexq.embedding(torch.zeros(2), wp, ws, 16, 128)
    with pytest.raises(ValueError, match="CUDA"):
        flexq.embedding(torch.zeros(2, dtype=torch.int64), wp, ws, 16, 128)
    with pytest.raises(ValueError, match="w must live"):
        flexq.quantize_weight4(torch.zeros(16, 256, dtype=torch.float16), 128)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        flexq.embedding_backward(x.float(), torch.zeros(2, dtype=torch.int64), wp, 16, 128)
