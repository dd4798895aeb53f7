"""4-bit layers on the GPU against the FP64 oracle: quantiser, read-back, matrix product."""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from w4_common import acts, layer, product_bound

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (3, 31), (17, 33), (40, 130), (33, 257), (16, 512), (130, 1000)]


# ---- quantiser and read-back ---------------------------------------------------------------
def _check_quantized(nq, W, group, d_in, symmetric, grid):
    q = nq.nq_w4_quantize(W.cuda(), group=group, d_in=None if d_in is None else d_in.cuda(),
                          symmetric=symmetric, grid=grid)
    m, n = W.shape
    codes, scales, zeros = O.quantize(W.double().numpy(), group,
                                      None if d_in is None else d_in.double().numpy(), symmetric, grid)
    np.testing.assert_array_equal(q["scales"].cpu().double().numpy(), scales)
    words = q["packed"].cpu().numpy().view(np.uint32)
    np.testing.assert_array_equal(words, O.pack(codes))        # codes past column n are 0
    if symmetric:
        assert q["zeros"] is None
    else:
        np.testing.assert_array_equal(q["zeros"].cpu().numpy(), zeros)
    ref = O.dequantize(codes, scales, zeros, group)
    out = nq.nq_w4_dequantize(q["packed"], q["scales"], n, group=group, zeros=q["zeros"])
    np.testing.assert_array_equal(out.cpu().double().numpy(), ref)       # exact in FP32
    out = nq.nq_w4_dequantize(q["packed"], q["scales"], n, group=group, zeros=q["zeros"],
                              dtype=torch.bfloat16)
    np.testing.assert_array_equal(out.cpu().double().numpy(), O.bf16(ref))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("m,n", SIZES)
def test_quantize_matches_the_oracle_exactly(nq, m, n, symmetric, dtype, group):
    rng = np.random.default_rng(m * 1000 + n)
    W = torch.from_numpy(0.02 * rng.standard_t(4, (m, n))).to(dtype)
    d = torch.from_numpy(np.exp(rng.standard_normal(n))).float()
    _check_quantized(nq, W, group, None, symmetric, 1)
    _check_quantized(nq, W, group, d, symmetric, 6)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_settles_halves_and_extremes_as_the_exact_quotient(nq, symmetric):
    # weights on and next to the halves of a step, tiny and huge scales, one-sided groups
    rows = []
    for e in (-126, -60, -3, 0, 60, 120):
        s = 2.0 ** e
        half = (np.arange(-13, 15, 2) / 2) * s
        near = np.concatenate([half, np.nextafter(half.astype(np.float32), np.float32(np.inf)),
                               np.nextafter(half.astype(np.float32), np.float32(-np.inf))])
        row = np.zeros(64)
        row[:len(near)] = near
        row[-2], row[-1] = -7 * s, 7 * s
        rows += [row, np.abs(row), -np.abs(row)]
    rows += [np.zeros(64), np.full(64, 2.0 ** -149), np.full(64, 3e38), -np.full(64, 1e-39),
             3e38 * np.linspace(-1, 1, 64)]
    W = torch.from_numpy(np.array(rows)).float()
    for grid in (1, 5):
        for group in (32, 64):
            _check_quantized(nq, W, group, None, symmetric, grid)


def test_quantize_with_extreme_importance(nq):
    # squares of d_in beyond FP32 range either way; the least error is still found
    rng = np.random.default_rng(9)
    W = torch.from_numpy(rng.standard_normal((8, 128))).float()
    for e in (-30, 30):
        d = torch.from_numpy(np.exp(rng.standard_normal(128)) * 10.0 ** e).float()
        _check_quantized(nq, W, 64, d, False, 16)
    _check_quantized(nq, W, 64, torch.zeros(128), True, 16)      # all errors 0: the first candidate


@pytest.mark.parametrize("symmetric", [True, False])
def test_a_weight_that_is_not_finite_spoils_its_own_group_only(nq, symmetric):
    rng = np.random.default_rng(4)
    W = torch.from_numpy(rng.standard_normal((3, 192))).float()
    clean = nq.nq_w4_quantize(W.cuda(), group=64, symmetric=symmetric, grid=3)
    ref = nq.nq_w4_dequantize(clean["packed"], clean["scales"], 192, 64, clean["zeros"]).cpu()
    bad = W.clone()
    bad[0, 70], bad[1, 5], bad[2, 191] = float("nan"), float("inf"), float("-inf")
    q = nq.nq_w4_quantize(bad.cuda(), group=64, symmetric=symmetric, grid=3)
    out = nq.nq_w4_dequantize(q["packed"], q["scales"], 192, 64, q["zeros"]).cpu()
    for i, g in ((0, 1), (1, 0), (2, 2)):
        assert out[i, 64 * g:64 * g + 64].isnan().all()
        ref[i, 64 * g:64 * g + 64] = out[i, 64 * g:64 * g + 64] = 0
    assert torch.equal(out, ref)


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_candidate_of_bf16_weights(nq, group, symmetric):
    # halves of a step, the type's extremes, zeros, subnormals; rows that end inside a word, a group
    # and a lane's columns; an infinite or NaN weight spoils its own group only
    rng = np.random.default_rng(group)
    step, n = 2.0 ** -4, 203
    halves = rng.choice(np.arange(-7, 7) + 0.5, size=n) * step
    halves[::8] = 7 * step
    rows = [halves, np.abs(halves), -np.abs(halves), np.zeros(n), np.full(n, 2.0 ** -133),
            3.3e38 * np.linspace(-1, 1, n), rng.standard_normal(n)]
    W = torch.from_numpy(np.array(rows)).to(torch.bfloat16)
    _check_quantized(nq, W, group, None, symmetric, 1)
    clean = nq.nq_w4_quantize(W.cuda(), group=group, symmetric=symmetric)
    ref = nq.nq_w4_dequantize(clean["packed"], clean["scales"], n, group, clean["zeros"]).cpu()
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = W.clone()
        bad[6, 40] = value
        q = nq.nq_w4_quantize(bad.cuda(), group=group, symmetric=symmetric)
        out = nq.nq_w4_dequantize(q["packed"], q["scales"], n, group, q["zeros"]).cpu()
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[6, 40 // group * group:min(n, (40 // group + 1) * group)] = True
        assert out[hit].isnan().all() and torch.equal(out[~hit], ref[~hit])


def test_quantize_of_a_view_that_starts_off_a_16_byte_boundary(nq):
    rng = np.random.default_rng(6)
    flat = torch.from_numpy(rng.standard_normal(1 + 5 * 64)).to(torch.bfloat16).cuda()
    W = flat[1:].view(5, 64)
    a, b = nq.nq_w4_quantize(W, group=32), nq.nq_w4_quantize(W.clone(), group=32)
    assert torch.equal(a["packed"], b["packed"]) and torch.equal(a["scales"], b["scales"])


# ---- matrix product --------------------------------------------------------------------------
def _check_product(nq, m, n, group, zeros, dtype, B, seed):
    What, (packed, scales, z) = layer(m, n, group, zeros, seed)
    X = acts(B, n, dtype, seed + 1)
    Y = nq.nq_w4_matmul(packed, scales, X.cuda(), group=group, zeros=z).cpu().double().numpy()
    Xd = X.double().numpy()
    err = np.abs(Y - O.matmul(Xd, What))
    assert (err <= product_bound(n) * O.matmul(np.abs(Xd), np.abs(What))).all()


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 2, 3, 7, 16, 17, 64, 65, 130, 300])
@pytest.mark.parametrize("m,n", SIZES)
def test_matmul_matches_the_oracle(nq, m, n, B, dtype, group, zeros):
    _check_product(nq, m, n, group, zeros, dtype, B, 7 * m + n + B)


@pytest.mark.parametrize("m,n,B", [(4096, 1024, 1), (300, 11008, 5), (1024, 4096, 16), (500, 8192, 200),
                                   (1000, 777, 513), (65, 28672, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_at_larger_sizes(nq, m, n, B, dtype):
    _check_product(nq, m, n, 128, False, dtype, B, 5)


@pytest.mark.parametrize("B", [1, 5, 40, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_of_small_integers_is_exact(nq, B, dtype):
    # codes times small whole numbers with power-of-two scales: every partial sum is exact
    rng = np.random.default_rng(B)
    m, n, g = 150, 333, 64
    codes, z = rng.integers(0, 16, (m, n)), rng.integers(0, 16, (m, 6))
    s = np.exp2(rng.integers(-2, 3, (m, 6)))
    X = rng.integers(-8, 9, (B, n)).astype(np.float64)
    dev = [torch.from_numpy(O.pack(codes).view(np.int32)).cuda(), torch.from_numpy(s).bfloat16().cuda()]
    Y = nq.nq_w4_matmul(*dev, torch.from_numpy(X).to(dtype).cuda(), group=g,
                        zeros=torch.from_numpy(z.astype(np.uint8)).cuda())
    np.testing.assert_array_equal(Y.cpu().double().numpy(), X @ O.dequantize(codes, s, z, g).T)


@pytest.mark.parametrize("B", [1, 24, 128])
def test_fp32_activations_keep_all_their_bits(nq, B):
    # one activation of 24 significant bits per row: the product of each of its three terms
    # is exact, and adding them rounds at most three times (half a step of 2^-23 each), the
    # scaling (three times) included: 6 * 2^-24 relative
    rng = np.random.default_rng(2)
    m, n = 200, 256
    What, (packed, scales, z) = layer(m, n, 128, True, 3)
    X = np.zeros((B, n), dtype=np.float32)
    at = rng.integers(0, n, B)
    X[np.arange(B), at] = rng.standard_normal(B).astype(np.float32) * np.exp2(rng.integers(-60, 60, B))
    Y = nq.nq_w4_matmul(packed, scales, torch.from_numpy(X).cuda(), group=128, zeros=z)
    ref = X.astype(np.float64) @ What.T
    assert (np.abs(Y.cpu().double().numpy() - ref) <= 6 * 2.0 ** -24 * np.abs(ref)).all()


@pytest.mark.parametrize("B", [1, 9, 70, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_do_not_touch_one_another(nq, B, dtype):
    # NaN and infinities in one row of X reach that row of Y alone; the others keep their bits
    What, (packed, scales, z) = layer(100, 320, 64, True, 8)
    X = acts(B, 320, dtype, 9).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z)
    bad = X.clone()
    bad[B // 2, 17], bad[B // 2, 200] = float("nan"), float("inf")
    out = nq.nq_w4_matmul(packed, scales, bad, group=64, zeros=z)
    assert out[B // 2].isnan().all()
    keep = torch.arange(B) != B // 2
    assert torch.equal(out[keep.cuda()], ref[keep.cuda()])


def test_largest_finite_activations_stay_finite(nq):
    packed = torch.from_numpy(O.pack(np.full((4, 32), 9)).view(np.int32)).cuda()     # q - 8 = 1
    scales = torch.full((4, 1), 0.25, dtype=torch.bfloat16, device="cuda")
    X = torch.zeros(2, 32, device="cuda")
    X[0, 3], X[1, 3] = torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max
    Y = nq.nq_w4_matmul(packed, scales, X, group=32)
    assert torch.equal(Y, X[:, 3:4].expand(2, 4) * 0.25)


def test_matmul_takes_vectors_views_and_a_workspace_of_the_user(nq):
    What, (packed, scales, z) = layer(50, 96, 32, False, 12)
    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.randn(1 + 3 * 96, device="cuda").to(dtype)
        X = flat[1:].view(3, 96)                    # not on a 16-byte boundary
        ref = nq.nq_w4_matmul(packed, scales, X.clone(), group=32)
        assert torch.equal(nq.nq_w4_matmul(packed, scales, X, group=32), ref)
        assert torch.equal(nq.nq_w4_matmul(packed, scales, X[1].clone(), group=32),
                           nq.nq_w4_matmul(packed, scales, X[1:2].clone(), group=32)[0])
        need = nq.lib.nq_w4_workspace_size(50, 96, nq.NQ_F32, 3)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(nq.nq_w4_matmul(packed, scales, X, group=32, ws=ws[:need]), ref)
        assert (ws[need:] == 255).all()


def test_wrappers_refuse_what_does_not_fit(nq):
    _, (packed, scales, z) = layer(8, 64, 32, True, 1)
    X = torch.zeros(2, 64, device="cuda")
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, X, group=48)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, X, group=64)                 # scales of another group size
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, torch.zeros(2, 65, device="cuda"), group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, X.t(), group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, X[:0], group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales.cpu(), X, group=32)
    with pytest.raises(TypeError):
        nq.nq_w4_matmul(packed, scales.float(), X, group=32)
    with pytest.raises(TypeError):
        nq.nq_w4_matmul(packed, scales, X.half(), group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, X, group=32, ws=torch.empty(64, device="cuda"))
    with pytest.raises(nq.NQError):
        nq.nq_w4_matmul(packed, scales, torch.zeros(99, 64, device="cuda"), group=32,
                        ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nq.NQError):
        nq.nq_w4_quantize(X, group=32, grid=0)
    with pytest.raises(ValueError):
        nq.nq_w4_quantize(X, group=32, d_in=torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        nq.nq_w4_dequantize(packed, scales, 64, group=32, dtype=torch.float16)


def test_calls_on_another_stream_and_in_a_graph(nq):
    What, (packed, scales, z) = layer(300, 1024, 128, True, 21)
    for dtype in (torch.float32, torch.bfloat16):
        for B in (2, 100):
            X = acts(B, 1024, dtype, 22).cuda()
            ref = nq.nq_w4_matmul(packed, scales, X, group=128, zeros=z)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                out = nq.nq_w4_matmul(packed, scales, X, group=128, zeros=z)
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(out, ref)
            static = torch.zeros_like(X)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = nq.nq_w4_matmul(packed, scales, static, group=128, zeros=z)
            for k in (1, 2):
                static.copy_(X * k)
                graph.replay()
                assert torch.equal(out, ref * k)


@pytest.mark.parametrize("B", [3, 40, 300])
def test_calls_on_two_streams_at_once(nq, B):
    What, (packed, scales, z) = layer(1000, 2048, 64, True, 23)
    X = acts(B, 2048, torch.float32, 24).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                out.append(nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in out)


def test_long_axis_and_many_rows(nq):
    # the longest k axis, on every path; more rows than one launch's worth of blocks
    _check_product(nq, 40, 65536, 128, True, torch.bfloat16, 2, 51)
    _check_product(nq, 40, 65536, 64, False, torch.bfloat16, 20, 52)
    _check_product(nq, 70000, 64, 32, True, torch.float32, 1, 53)
    _check_product(nq, 70000, 64, 32, False, torch.bfloat16, 33, 54)


def test_repeated_calls_give_the_same_bits(nq):
    What, (packed, scales, z) = layer(700, 3000, 128, True, 61)
    for B in (1, 7, 16, 90):
        for dtype in (torch.float32, torch.bfloat16):
            X = acts(B, 3000, dtype, 62).cuda()
            ref = nq.nq_w4_matmul(packed, scales, X, group=128, zeros=z)
            for _ in range(5):
                assert torch.equal(nq.nq_w4_matmul(packed, scales, X, group=128, zeros=z), ref)


def test_zero_points_past_4_bits_count_by_their_low_bits(nq):
    What, (packed, scales, z) = layer(60, 512, 64, True, 71)
    X = acts(20, 512, torch.bfloat16, 72).cuda()
    for x in (X[:2].contiguous(), X):
        assert torch.equal(nq.nq_w4_matmul(packed, scales, x, group=64, zeros=z + 48),
                           nq.nq_w4_matmul(packed, scales, x, group=64, zeros=z))
    assert torch.equal(nq.nq_w4_dequantize(packed, scales, 512, 64, z + 48),
                       nq.nq_w4_dequantize(packed, scales, 512, 64, z))


def test_scales_that_start_off_a_word(nq):
    # a row slice of a larger layer: scales and zero points at any address
    What, (packed, scales, z) = layer(65, 768, 128, True, 81)
    X = acts(30, 768, torch.float32, 82).cuda()
    for x in (X[:1].contiguous(), X[:4].contiguous(), X):
        ref = nq.nq_w4_matmul(packed, scales, x, group=128, zeros=z)
        flat_s = torch.cat([scales.new_zeros(1), scales.flatten()])[1:].view(65, -1)
        flat_z = torch.cat([z.new_zeros(1), z.flatten()])[1:].view(65, -1)
        assert torch.equal(nq.nq_w4_matmul(packed, flat_s, x, group=128, zeros=flat_z), ref)
        assert torch.equal(nq.nq_w4_matmul(packed[1:], scales[1:], x, group=128, zeros=z[1:]),
                           ref[:, 1:])


def test_from_calibration_to_a_quantised_layer(nq):
    # calibration -> quantiser weighted by d_in -> product: the search lowers the weighted
    # error, and the layer applies as what it reads back
    rng = np.random.default_rng(31)
    m, n, T = 256, 384, 2048
    W = torch.from_numpy(0.02 * rng.standard_t(3, (m, n))).float().cuda()
    scale = torch.from_numpy(np.exp(rng.standard_normal(n))).float().cuda()
    A = torch.randn(T, n, device="cuda") * scale
    d_in, _, _, _ = nq.nq_calib_precond(A, torch.randn(T, m, device="cuda"))
    errs = []
    for grid in (1, 16):
        q = nq.nq_w4_quantize(W, group=64, d_in=d_in, symmetric=False, grid=grid)
        Wq = nq.nq_w4_dequantize(q["packed"], q["scales"], n, group=64, zeros=q["zeros"])
        errs.append(float((((W - Wq) * d_in).double() ** 2).sum()))
        X = A[:5].contiguous()
        Y = nq.nq_w4_matmul(q["packed"], q["scales"], X, group=64, zeros=q["zeros"])
        ref = X.double() @ Wq.double().T
        bound = product_bound(n) * (X.double().abs() @ Wq.double().abs().T)
        assert ((Y.double() - ref).abs() <= bound).all()
    assert errs[1] < errs[0]
