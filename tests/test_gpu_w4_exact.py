"""Long axes, split axes and many tiles of the 4-bit products, where every sum is exact in FP32.

A bound that grows with the length of the axis lets a missing part of a long one pass; equality does
not.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from w4_exact import assert_exact, dense, layer, wide

pytestmark = pytest.mark.gpu


def _check(nq, W, dev, group, X, dtype, least):
    assert_exact(X, W, least)
    Y = nq.nq_w4_matmul(dev[0], dev[1], torch.from_numpy(X).to(dtype).cuda(), group=group, zeros=dev[2])
    np.testing.assert_array_equal(Y.cpu().double().numpy(), X @ W.T)


# the k axis over eight warps (columns in shared memory, then from global memory), and in parts over
# the SMs with more than 16 columns
@pytest.mark.parametrize("n", [4173, 11008, 28672, 65536])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_axes(nq, n, dtype, group, zeros):
    W, dev = layer(65, n, group, zeros, n + group, 0, 2)
    for B in (1, 2, 5, 16, 17, 40, 130):
        _check(nq, W, dev, group, dense(B, n, B), dtype, 1)


@pytest.mark.parametrize("n", [300, 4173, 11008, 65536])
@pytest.mark.parametrize("group,zeros", [(32, False), (128, True)])
def test_all_terms_of_fp32_activations_along_the_axis(nq, n, group, zeros):
    # a hundred rows of X, four places each: every range of the axis, and most units of the longest
    W, dev = layer(33, n, group, zeros, n + group, 0, 1)
    X = wide(100, n, n)
    _check(nq, W, dev, group, X, torch.float32, 1)
    for B in (1, 4, 5):
        for b in range(0, 100 - B, 25):
            _check(nq, W, dev, group, X[b:b + B], torch.float32, 1)


# more tiles than SMs, several stages each: the rings carry on from tile to tile
@pytest.mark.parametrize("m,B", [(25600, 20), (20000, 50), (6000, 513)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, True), (128, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_tiles_an_sm(nq, m, B, dtype, group, zeros):
    W, dev = layer(m, 1100, group, zeros, m + group)
    _check(nq, W, dev, group, dense(B, 1100, B), dtype, 0.25)


# many jobs a CTA of the product for few columns
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_jobs_a_cta(nq, dtype, group, zeros):
    for m, n in ((40000, 600), (9000, 4173)):
        W, dev = layer(m, n, group, zeros, m)
        for B in (1, 5, 16):
            _check(nq, W, dev, group, dense(B, n, B), dtype, 0.25)


@pytest.mark.parametrize("n,B,dtype", [(11008, 5, torch.float32), (11008, 3, torch.bfloat16),
                                       (4173, 20, torch.bfloat16), (4173, 200, torch.float32),
                                       (777, 33, torch.float32)])
def test_a_call_stays_inside_its_workspace(nq, n, B, dtype):
    W, dev = layer(150, n, 64, True, 4, 0, 2)
    X = dense(B, n, 5)
    need = nq.lib.nq_w4_workspace_size(150, n, nq.NQ_BF16 if dtype == torch.bfloat16 else nq.NQ_F32, B)
    assert need > 0
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    Y = nq.nq_w4_matmul(dev[0], dev[1], torch.from_numpy(X).to(dtype).cuda(), group=64, zeros=dev[2],
                        ws=ws[:need])
    np.testing.assert_array_equal(Y.cpu().double().numpy(), X @ W.T)
    assert (ws[need:] == 171).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_most_rows_of_x_and_of_w(nq, dtype):
    W, dev = layer(200, 300, 64, True, 7)
    _check(nq, W, dev, 64, dense(65536, 300, 8), dtype, 0.25)
    m = 1 << 24
    packed = torch.randint(-2 ** 31, 2 ** 31, (m, 4), dtype=torch.int32, device="cuda")
    scales = torch.ones(m, 1, dtype=torch.bfloat16, device="cuda")
    at = torch.cat([torch.arange(300), torch.arange(m - 300, m)]).cuda()
    W = torch.from_numpy(O.unpack(packed[at].cpu().numpy().view(np.uint32), 31) - 8).double()
    for B in (2, 17):
        X = dense(B, 31, B)
        Y = nq.nq_w4_matmul(packed, scales, torch.from_numpy(X).to(dtype).cuda(), group=32)
        np.testing.assert_array_equal(Y[:, at].cpu().double().numpy(), X @ W.numpy().T)


def test_more_than_2_to_the_32_words_of_codes(nq):
    m, n, last = (1 << 21) + 200, 16384, 300
    packed = torch.empty(m, n // 8, dtype=torch.int32, device="cuda")
    for i in range(0, m, 1 << 19):
        part = packed[i:i + (1 << 19)]
        part.copy_(torch.randint(-2 ** 31, 2 ** 31, part.shape, dtype=torch.int32, device="cuda"))
    assert packed.numel() > 2 ** 32
    scales = torch.ones(m, n // 128, dtype=torch.bfloat16, device="cuda")
    W = O.unpack(packed[-last:].cpu().numpy().view(np.uint32), n) - 8.0
    for B in (1, 16, 20):
        X = dense(B, n, B)
        assert_exact(X, W, 1)
        Y = nq.nq_w4_matmul(packed, scales, torch.from_numpy(X).bfloat16().cuda(), group=128)
        np.testing.assert_array_equal(Y[:, -last:].cpu().double().numpy(), X @ W.T)


def test_more_than_2_to_the_32_weights(nq):
    m, n, last = (1 << 18) + 100, 16384, 200
    W = torch.empty(m, n, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02)
    assert W.numel() > 2 ** 32
    tail = W[-last:].clone()
    for symmetric, grid in ((True, 1), (False, 3)):
        q = nq.nq_w4_quantize(W, group=128, symmetric=symmetric, grid=grid)
        t = nq.nq_w4_quantize(tail, group=128, symmetric=symmetric, grid=grid)
        for k in ("packed", "scales") + (() if symmetric else ("zeros",)):
            assert torch.equal(q[k][-last:], t[k])
        out = nq.nq_w4_dequantize(q["packed"], q["scales"], n, 128, q["zeros"], dtype=torch.bfloat16)
        assert torch.equal(out[-last:], nq.nq_w4_dequantize(t["packed"], t["scales"], n, 128, t["zeros"],
                                                            dtype=torch.bfloat16))
        del out
