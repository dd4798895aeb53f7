"""4-bit layers whose products are exact in FP32: whole codes and activations, power-of-two scales.

Every partial sum is then a whole number of the least scale, and below 2^24 of them no addition
rounds, whatever its order (``assert_exact`` holds the inputs to that).  So a result has to be equal
to the FP64 one, and a part of the k axis that is left out, or taken twice, shows however long it is.
"""
import numpy as np
import torch

from oracle import w4 as O


def to_gpu(codes, scales, zeros):
    return (torch.from_numpy(O.pack(codes).view(np.int32)).cuda(),
            torch.from_numpy(scales).to(torch.bfloat16).cuda(),
            None if zeros is None else torch.from_numpy(zeros.astype(np.uint8)).cuda())


def layer(m, n, group, zeros, seed, low=-2, high=3):
    """(W^ float64, (packed, scales, zeros) on the GPU); scales 2^low .. 2^(high - 1)."""
    rng = np.random.default_rng(seed)
    ng = -(-n // group)
    codes = rng.integers(0, 16, (m, n), dtype=np.int8)
    s = np.exp2(rng.integers(low, high, (m, ng)))
    z = rng.integers(0, 16, (m, ng)) if zeros else None
    return O.dequantize(codes, s, z, group), to_gpu(codes, s, z)


def assert_exact(X, W, least):
    """No sum of |W x| passes 2^24 units of the least scale."""
    assert (np.abs(X) @ np.abs(W).T).max() / least < 2 ** 24


def dense(B, n, seed):
    return np.random.default_rng(seed).integers(-8, 9, (B, n)).astype(np.float64)


def wide(B, n, seed):
    """Four activations a row that need all three BF16 terms of an FP32 value, in different places."""
    rng = np.random.default_rng(seed)
    X = np.zeros((B, n))
    for b in range(B):
        at = rng.choice(n, min(4, n), replace=False)
        X[b, at] = rng.integers(2 ** 16, 2 ** 17, len(at)) * rng.choice([-1, 1], len(at))
    return X
