"""Products of 4-bit layers at the ends of FP32's range, and with scales that are not finite."""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from w4_common import acts, layer, product_bound
from w4_exact import to_gpu

pytestmark = pytest.mark.gpu

FP32_MAX = float(torch.finfo(torch.float32).max)
BF16_MAX = float(torch.finfo(torch.bfloat16).max)

# (n, B): columns in shared memory, columns from global memory, tcgen05, tcgen05 with the k axis split
PATHS = [(200, 1), (200, 5), (12000, 2), (12000, 5), (200, 24), (12000, 24), (200, 200)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,B", PATHS)
def test_products_stay_finite_where_the_result_does(nq, n, B, dtype, group):
    # every activation the type's largest or its negative, all codes, zero points from end to end:
    # one product alone passes the range before its scale, and so does a group's sum
    rng = np.random.default_rng(n + B + group)
    m, ng = 40, -(-n // group)
    z = np.tile([0, 15, 8, 3], (m, ng))[:, :ng]
    codes = rng.integers(0, 16, (m, n))
    codes[0], codes[1] = 15, 0                                # every sum at its largest
    s = np.full((m, ng), 2.0 ** -19)                          # 12000 x 15 x 2^-19 < 0.35
    What = O.dequantize(codes, s, z, group)
    big = FP32_MAX if dtype == torch.float32 else BF16_MAX
    X = np.where(rng.random((B, n)) < 0.5, big, -big)
    X[0] = big
    Y = nq.nq_w4_matmul(*to_gpu(codes, s, z)[:2], torch.from_numpy(X).to(dtype).cuda(), group=group,
                        zeros=torch.from_numpy(z.astype(np.uint8)).cuda()).cpu().double().numpy()
    assert np.isfinite(Y).all()
    err = np.abs(Y / big - (X / big) @ What.T)
    assert (err <= product_bound(n) * (np.abs(X / big) @ np.abs(What).T)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 9])
def test_an_expert_whose_up_projection_nears_the_range(nq, B, dtype):
    # gate rows of zeros: h = 0 times an up projection that is finite (7 x 2^-8 of the largest
    # value), although 7 / 4 of it is not
    d, f = 96, 40
    codes = np.full((2 * f, d), 8)
    codes[f:, 5] = 15
    gu = to_gpu(codes, np.full((2 * f, 3), 2.0 ** -8), None)
    dn = to_gpu(np.full((d, f), 9), np.full((d, 2), 1.0), None)
    X = torch.zeros(B, d, dtype=dtype)
    X[:, 5] = torch.finfo(dtype).max
    Y = nq.nq_moe_w4(X.cuda(), torch.zeros(1, d, dtype=dtype, device="cuda"), gu[0][None], gu[1][None],
                     dn[0][None], dn[1][None], 1, group=32)
    assert torch.equal(Y.cpu(), torch.zeros(B, d))


@pytest.mark.parametrize("B", [1, 5, 24, 100])
@pytest.mark.parametrize("e", [-110, -100, -80])
def test_small_fp32_activations_keep_their_bits(nq, B, e):
    # one activation of 24 significant bits per row: its three products are exact, and what follows
    # (three scalings, up to nine additions) rounds at most twelve times: 6 units of 2^-23 of the
    # result, or, where the sum in units of 2^-11 is subnormal, 12 halves of 2^-149 2^11
    rng = np.random.default_rng(B - e)
    m, n = 100, 256
    What, (packed, scales, z) = layer(m, n, 64, True, 3)
    X = np.zeros((B, n), dtype=np.float32)
    X[np.arange(B), rng.integers(0, n, B)] = np.ldexp(rng.uniform(1, 2, B).astype(np.float32), e)
    Y = nq.nq_w4_matmul(packed, scales, torch.from_numpy(X).cuda(), group=64, zeros=z)
    ref = X.astype(np.float64) @ What.T
    err = np.abs(Y.cpu().double().numpy() - ref)
    assert (err <= 6 * 2.0 ** -23 * np.abs(ref) + 12 * 2.0 ** -139).all()


@pytest.mark.parametrize("group,n", [(32, 33), (64, 200), (128, 1100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 5, 24, 100])
def test_a_scale_that_is_not_finite_reaches_its_own_row_alone(nq, B, dtype, group, n):
    What, (packed, scales, z) = layer(20, n, group, True, 5)
    X = acts(B, n, dtype, 6).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=group, zeros=z)
    bad = scales.clone()
    bad[3, 0], bad[7, -1] = float("nan"), float("nan")
    bad[11, 0], bad[19, -1] = float("inf"), float("inf")
    Y = nq.nq_w4_matmul(packed, bad, X, group=group, zeros=z)
    assert Y[:, [3, 7]].isnan().all() and not Y[:, [11, 19]].isfinite().any()
    keep = [i for i in range(20) if i not in (3, 7, 11, 19)]
    assert torch.equal(Y[:, keep], ref[:, keep])
