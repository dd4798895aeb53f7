"""Layers with 4-bit weights and group scales, FP64 oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Format of an m x n layer with group size g: codes 0..15 packed eight to a 32-bit word, code
of column k in nibble k % 8 (lowest first) of word k // 8, rows of 4 ceil(n / 32) words; a
scale (a BF16 value) and a zero point per row and group;  W^ = scale (code - zero).
"""
import numpy as np


def bf16(x):
    """x rounded to FP32 and then to BF16 (both to nearest, ties to even), as float64."""
    b = np.ascontiguousarray(np.asarray(x, dtype=np.float32)).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)).astype(np.uint32)
    return r.view(np.float32).astype(np.float64).reshape(np.shape(x))


def group_of(n, group):
    return np.arange(n) // group


def pack(codes):
    m, n = codes.shape
    ld = 4 * -(-n // 32)
    full = np.zeros((m, 8 * ld), dtype=np.uint32)
    full[:, :n] = codes
    return np.bitwise_or.reduce(full.reshape(m, ld, 8) << (4 * np.arange(8, dtype=np.uint32)), axis=2)


def unpack(words, n):
    words = np.asarray(words, dtype=np.uint32)
    codes = (words[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    return codes.reshape(words.shape[0], -1)[:, :n].astype(np.int64)


def _candidate(w, alpha, symmetric):
    """Scale, zero point and codes of one group of finite weights at clipping alpha."""
    if symmetric:
        s, z = float(bf16(alpha * np.max(np.abs(w)) / 7)), 8.0
    else:
        lo, hi = min(0.0, np.min(w)), max(0.0, np.max(w))
        s = float(bf16(alpha * (hi - lo) / 15))
        z = float(np.clip(np.rint(-alpha * lo / s), 0, 15)) if s > 0 else 0.0
    q = np.clip(np.rint(w / s) + z, 0, 15) if s > 0 else np.full(len(w), z)
    return s, z, q


def quantize(W, group, d_in=None, symmetric=True, grid=1):
    """codes (m, n), scales and zeros (m, groups) of the least weighted squared error over the
    candidates alpha = 1 - c / (2 grid); the lowest c wins a tie."""
    W = np.asarray(W, dtype=np.float64)
    m, n = W.shape
    d = np.ones(n) if d_in is None else np.asarray(d_in, dtype=np.float64)
    ng = -(-n // group)
    codes = np.zeros((m, n), dtype=np.int64)
    scales, zeros = np.zeros((m, ng)), np.zeros((m, ng), dtype=np.int64)
    for i in range(m):
        for j in range(ng):
            c = slice(j * group, min(n, (j + 1) * group))
            w = W[i, c]
            best = None
            for t in range(grid):
                s, z, q = _candidate(w, 1 - t / (2 * grid), symmetric)
                err = np.sum((d[c] * (w - s * (q - z))) ** 2)
                if best is None or err < best[0]:
                    best = (err, s, z, q)
            scales[i, j], zeros[i, j], codes[i, c] = best[1], best[2], best[3]
    return codes, scales, zeros


def dequantize(codes, scales, zeros, group):
    """W^; zeros None means 8."""
    g = group_of(codes.shape[-1], group)
    z = 8 if zeros is None else np.asarray(zeros)[..., g]
    return np.asarray(scales, dtype=np.float64)[..., g] * (codes - z)


def matmul(X, What):
    return np.asarray(X, dtype=np.float64) @ What.T


def silu(v):
    return v / (1 + np.exp(-v))


def route(X, router, top_k, renormalise):
    """ids and weights of the chosen experts by falling logit, ties to the lowest expert."""
    logits = np.asarray(X, dtype=np.float64) @ np.asarray(router, dtype=np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    top = np.take_along_axis(logits, ids, 1)
    over = top if renormalise else logits
    peak = top[:, :1]
    return ids, np.exp(top - peak) / np.exp(over - peak).sum(1, keepdims=True)


def moe(X, router, gate_up, down, top_k, renormalise=True):
    """y, ids, weights of the layer; gate_up (E, 2f, d) and down (E, d, f) dense."""
    X = np.asarray(X, dtype=np.float64)
    ids, p = route(X, router, top_k, renormalise)
    f = gate_up.shape[1] // 2
    Y = np.zeros((X.shape[0], down.shape[1]))
    for b in range(X.shape[0]):
        for j in range(top_k):
            gu = gate_up[ids[b, j]] @ X[b]
            Y[b] += p[b, j] * (down[ids[b, j]] @ (silu(gu[:f]) * gu[f:]))
    return Y, ids, p
