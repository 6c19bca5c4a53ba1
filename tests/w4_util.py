"""Plain numpy forms of the 4-bit weights and of the table operators, in 64
bits (test infrastructure; shares no code with the library)."""

import numpy as np
import torch


def quantize4(w16, gs):
    """Codes int8 [N, K] and FP16 scales [N, G] of FP16 weights."""
    g = w16.astype(np.float64).reshape(w16.shape[0], -1, gs)
    s = (np.abs(g).max(-1).astype(np.float32) / np.float32(7)).astype(np.float16)
    s32 = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(g.astype(np.float32) / s32)
    q = np.where(s32 > 0, np.clip(np.where(np.isfinite(q), q, 0), -7, 7), 0)
    return q.reshape(w16.shape).astype(np.int8), s


NIBBLES = (0, 4, 2, 6, 1, 5, 3, 7)           # of a word's eight columns


def pack4(q):
    """The packed bytes of codes [N, K] in -8 .. 7."""
    N, K = q.shape
    Np, Kp = -(-N // 16) * 16, -(-K // 128) * 128
    u = np.full((Np, Kp), 8, dtype=np.uint32)
    u[:N, :K] = q.astype(np.int64) + 8
    # [row tile, row, column tile, word, chunk, column of the word]
    u = u.reshape(Np // 16, 16, Kp // 128, 4, 4, 8)
    words = np.zeros(u.shape[:-1], dtype=np.uint32)
    for i in range(8):
        words |= u[..., i] << np.uint32(4 * NIBBLES[i])
    # -> [row tile, column tile, row, chunk, word]
    return np.ascontiguousarray(words.transpose(0, 2, 1, 4, 3)).astype("<u4").view(np.uint8).reshape(-1)


def unpack4(b, N, K):
    """The codes [N, K] of packed bytes."""
    rt, ct = -(-N // 16), -(-K // 128)
    words = b.view("<u4").reshape(rt, ct, 16, 4, 4).transpose(0, 2, 1, 4, 3)
    q = np.stack([(words >> np.uint32(4 * NIBBLES[i])) & 15 for i in range(8)], axis=-1)
    return (q.astype(np.int64) - 8).astype(np.int8).reshape(rt * 16, ct * 128)[:N, :K]


def dequantize(q, s):
    """FP64 [N, K] of codes and scales [N, G]."""
    gs = q.shape[1] // s.shape[1]
    return q.astype(np.float64) * np.repeat(s.astype(np.float64), gs, axis=1)


def to64(t):
    return t.detach().cpu().double().numpy()


def embedding64(ids, w64, scale):
    ids = np.asarray(ids).reshape(-1)
    out = np.zeros((ids.size, w64.shape[1]))
    here = (ids >= 0) & (ids < w64.shape[0])
    out[here] = w64[ids[here]] * scale
    return out


def embedding_backward64(dy, ids, q, gs, scale):
    """(D [V, K], ds [V, G]) in 64 bits."""
    ids = np.asarray(ids).reshape(-1)
    D = np.zeros(q.shape)
    here = (ids >= 0) & (ids < q.shape[0])
    np.add.at(D, ids[here], dy.reshape(ids.size, -1)[here] * scale)
    ds = (D * q).reshape(q.shape[0], -1, gs).sum(-1)
    return D, ds


def half_step(t):
    """Half a rounding step of a type, relative to the value."""
    return torch.finfo(t).eps / 2
