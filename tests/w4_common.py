"""Seeded 4-bit layers for the tests, on the CPU (oracle form) and on the GPU."""
import numpy as np
import torch

from oracle import w4 as O


def layer(rows, n, group, zeros, seed, scale=0.01):
    """(What float64 (rows, n), (packed, scales, zeros) on the GPU) of random codes.

    The codes past column n are random too: they must not matter.
    """
    rng = np.random.default_rng(seed)
    ld, ng = 4 * -(-n // 32), -(-n // group)
    full = rng.integers(0, 16, (rows, 8 * ld))
    scales = O.bf16(scale * np.exp(0.5 * rng.standard_normal((rows, ng))))
    z = rng.integers(0, 16, (rows, ng)) if zeros else None
    dev = (torch.from_numpy(O.pack(full).view(np.int32)).cuda(),
           torch.from_numpy(scales).to(torch.bfloat16).cuda(),
           torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None)
    return O.dequantize(full[:, :n], scales, z, group), dev


def stack(E, rows, n, group, zeros, seed, scale=0.01):
    """E layers as one array each: (E, rows, .) on both sides."""
    What, dev = layer(E * rows, n, group, zeros, seed, scale)
    return What.reshape(E, rows, n), tuple(None if t is None else t.view(E, rows, -1) for t in dev)


def acts(B, n, dtype, seed):
    x = np.random.default_rng(seed).standard_normal((B, n))
    return torch.from_numpy(x).to(dtype)


# Bound of the products' error relative to sum_k |W^_ik x_k|: exact products, and at most
# (all terms counted one after another) n additions inside the tensor-core instructions and
# n / 32 + 40 outside (groups, warps, terms), each off by at most one unit of 2^-23 (twice a
# rounding to nearest: the instructions may truncate) of a partial sum that the sum of
# magnitudes bounds.
def product_bound(n):
    return (n + n / 32 + 40) * 2.0 ** -23
