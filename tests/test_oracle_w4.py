"""The 4-bit oracle against closed forms and direct restatements."""
import numpy as np
import pytest
import torch

from oracle import w4


def test_bf16_rounding_matches_torch():
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 10.0 ** np.arange(-20, 20).repeat(100),
                        [0.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 2.0 ** -133, 3e38]])
    ref = torch.from_numpy(x).float().bfloat16().double().numpy()
    np.testing.assert_array_equal(w4.bf16(x), ref)


@pytest.mark.parametrize("n", [1, 7, 8, 31, 32, 33, 100])
def test_pack_round_trip_and_word_layout(n):
    codes = np.random.default_rng(n).integers(0, 16, (5, n))
    words = w4.pack(codes)
    assert words.shape == (5, 4 * -(-n // 32))
    np.testing.assert_array_equal(w4.unpack(words, n), codes)
    for k in range(n):
        np.testing.assert_array_equal((words[:, k // 8] >> np.uint32(4 * (k % 8))) & 15, codes[:, k])


@pytest.mark.parametrize("symmetric", [True, False])
def test_values_on_the_grid_are_recovered_exactly(symmetric):
    # with a power-of-two scale and the extreme codes present, rounding gives the codes back
    rng = np.random.default_rng(1)
    n, g = 96, 32
    if symmetric:
        q = rng.integers(1, 16, (4, n))
        q[:, ::g] = 15               # |w| = 7 s: s = max / 7 exactly
        z = np.full((4, n // g), 8)
    else:
        q = rng.integers(0, 16, (4, n))
        q[:, ::g], q[:, 1::g] = 0, 15
        z = rng.integers(0, 16, (4, n // g))
    s = np.exp2(rng.integers(-8, 3, (4, n // g)))
    W = w4.dequantize(q, s, z, g)
    codes, scales, zeros = w4.quantize(W, g, symmetric=symmetric)
    np.testing.assert_array_equal(codes, q)
    np.testing.assert_array_equal(scales, s)
    np.testing.assert_array_equal(zeros, z)


def test_ties_go_to_even_and_zero_groups_to_zero():
    s = 0.5
    w = np.zeros((1, 32))
    w[0, :5] = np.array([7, 0.5, 1.5, -0.5, -2.5]) * s
    codes, scales, zeros = w4.quantize(w, 32)
    assert scales[0, 0] == s
    np.testing.assert_array_equal(codes[0, :5] - 8, [7, 0, 2, 0, -2])
    codes, scales, zeros = w4.quantize(np.zeros((1, 40)), 32, symmetric=False)
    assert not scales.any() and not w4.dequantize(codes, scales, zeros, 32).any()


def test_search_never_increases_the_weighted_error():
    rng = np.random.default_rng(3)
    W, d = rng.standard_t(3, (6, 130)), np.exp(rng.standard_normal(130))
    for symmetric in (True, False):
        errs = []
        for grid in (1, 2, 4, 8):     # each grid's candidates contain the one before's
            c, s, z = w4.quantize(W, 64, d, symmetric, grid)
            errs.append((((W - w4.dequantize(c, s, z, 64)) * d) ** 2).sum())
        assert all(b <= a for a, b in zip(errs, errs[1:]))
        assert errs[-1] < errs[0]


@pytest.mark.parametrize("renormalise", [True, False])
def test_moe_matches_a_direct_sum_over_all_experts(renormalise):
    rng = np.random.default_rng(5)
    E, d, f, B, k = 6, 10, 7, 4, 3
    X, R = rng.standard_normal((B, d)), rng.standard_normal((E, d))
    GU, D = rng.standard_normal((E, 2 * f, d)), rng.standard_normal((E, d, f))
    Y, ids, p = w4.moe(X, R, GU, D, k, renormalise)
    logits = X @ R.T
    soft = np.exp(logits) / np.exp(logits).sum(1, keepdims=True)
    for b in range(B):
        y, kept = np.zeros(d), 0.0
        for e in range(E):
            if (logits[b] > logits[b, e]).sum() >= k:     # not among the k largest
                continue
            g, u = GU[e, :f] @ X[b], GU[e, f:] @ X[b]
            y += soft[b, e] * (D[e] @ (g / (1 + np.exp(-g)) * u))
            kept += soft[b, e]
        np.testing.assert_allclose(Y[b], y / kept if renormalise else y, rtol=1e-12)


def test_equal_logits_choose_the_lowest_experts():
    X, R = np.ones((1, 4)), np.ones((5, 4))
    R[3] = 2
    ids, p = w4.route(X, R, 3, True)
    np.testing.assert_array_equal(ids, [[3, 0, 1]])
