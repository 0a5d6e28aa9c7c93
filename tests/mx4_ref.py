"""Plain 64-bit restatement of the MXFP4 format and the expert operators, for the
tests only: numpy, one definition at a time, no blocking and no packing."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes [M, K / 2], scale bytes [M, K / 32]) of float64 rows."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    b = np.where(finite[:, :, None], b, 0.0)
    amax = np.abs(b).max(axis=2)
    e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.minimum(np.abs(b) / np.exp2(e.astype(np.float64))[:, :, None], 6.0)
    d = np.abs(a[..., None] - LEVELS)                       # distance to every level
    near = d.min(axis=-1, keepdims=True)
    even = np.arange(8) % 2 == 0
    code = np.argmax((d == near) * (1.0 + even), axis=-1)   # nearest; at a tie the even code
    code = (code + 8 * np.signbit(b)).reshape(M, K // 2, 2).astype(np.uint8)
    scale = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale


def values(codes, scale):
    """float64 values [..., K] of codes [..., K / 2] and scale bytes [..., K / 32]."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*scale.shape, 32)
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127.0))
    v = np.where(c >= 8, -1.0, 1.0) * LEVELS[c & 7] * s[..., None]
    return v.reshape(*scale.shape[:-1], scale.shape[-1] * 32)


def words(scale):
    """Row-major scale bytes [M, K / 32] in the words layout [ceil(K / 128), M, 4]."""
    M, n = scale.shape
    p = np.zeros((M, -(-n // 4) * 4), np.uint8)
    p[:, :n] = scale
    return np.ascontiguousarray(p.reshape(M, -1, 4).transpose(1, 0, 2))


def rows_of_words(w, K):
    return np.ascontiguousarray(w.transpose(1, 0, 2).reshape(w.shape[1], -1)[:, :K // 32])


def gemm(x, w):
    """(y, tolerance) in float64. A product of two codes and two scales is exact in fp32; one fp32 addition per 64
    columns (and one per partial sum joined, at most 8) is off by at most 2^-23 of the magnitudes summed; the bf16
    result by half a step, 2^-8 of it, plus half the smallest step where it is subnormal."""
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    acc = (-(-x.shape[1] // 64) + 8) * 2.0 ** -23 * mag
    return y, (np.abs(y) + acc) * 2.0 ** -8 + acc + 2.0 ** -134


def sort(ids, E):
    M, k = ids.shape
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < E)
    order = [i for e in range(E) for i in np.flatnonzero(flat == e)]
    offsets = np.concatenate(([0], np.cumsum([(flat[live] == e).sum() for e in range(E)]))).astype(np.int32)
    rows, pos = np.full(M * k, -1, np.int32), np.full(M * k, -1, np.int32)
    for slot, i in enumerate(order):
        rows[slot], pos[i] = i // k, slot
    return offsets, rows, pos.reshape(M, k)


def combine(y, pos, weights):
    """(out, tolerance): k products and additions in fp32 (2^-24 each, of the magnitudes summed), one bf16 rounding."""
    T = y.shape[0]
    live = (pos >= 0) & (pos < T)
    rows = y[np.where(live, pos, 0)] if T else np.zeros((*pos.shape, y.shape[1]))
    t = np.where(live[:, :, None], np.where(live, weights, 0.0)[:, :, None] * np.where(live[:, :, None], rows, 0.0), 0.0)
    out, mag = t.sum(axis=1), np.abs(t).sum(axis=1)
    acc = (pos.shape[1] + 1) * 2.0 ** -24 * mag
    return out, (np.abs(out) + acc) * 2.0 ** -8 + acc + 2.0 ** -134
