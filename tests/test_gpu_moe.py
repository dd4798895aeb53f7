"""Mixture-of-experts layer on 4-bit experts against the FP64 oracle."""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from w4_common import acts, layer, product_bound, stack

pytestmark = pytest.mark.gpu


def _setup(B, E, d, f, group, zeros, dtype, seed):
    GU, gu = stack(E, 2 * f, d, group, zeros, seed, scale=0.15 / np.sqrt(d))
    D, dn = stack(E, d, f, group, zeros, seed + 1, scale=0.15 / np.sqrt(f))
    X = acts(B, d, dtype, seed + 2)
    R = (acts(E, d, torch.float64, seed + 3) / np.sqrt(d)).to(dtype)
    return GU, gu, D, dn, X, R


def _run(nq, X, R, gu, dn, k, group, renormalise, **kw):
    return nq.nq_moe_w4(X.cuda(), R.cuda(), gu[0], gu[1], dn[0], dn[1], k, group=group,
                        gate_up_zeros=gu[2], down_zeros=dn[2], renormalise=renormalise, **kw)


def _y_bound(X, GU, D, ids, p):
    """Elementwise error bound of Y, from the products' bound: with g and u off by at most dg
    and du, h = silu(g) u is off by 1.1 dg |u| + |silu(g)| du + dg du (|silu'| <= 1.1) and by
    8 roundings of its own (exp, quotient, products); y by its products' bound, by D times
    that, and by 4 roundings per summand (weight included)."""
    B, k = ids.shape
    f = GU.shape[1] // 2
    out = np.zeros((B, D.shape[1]))
    for b in range(B):
        for j in range(k):
            W, Dn = GU[ids[b, j]], D[ids[b, j]]
            gu = W @ X[b]
            e = product_bound(W.shape[1]) * (np.abs(W) @ np.abs(X[b]))
            g, u, dg, du = gu[:f], gu[f:], e[:f], e[f:]
            h = np.abs(O.silu(g) * u)
            dh = 1.1 * dg * np.abs(u) + np.abs(O.silu(g)) * du + dg * du + 8 * 2.0 ** -23 * h
            mag = np.abs(Dn) @ h
            out[b] += p[b, j] * (np.abs(Dn) @ dh + (product_bound(f) + (4 + k) * 2.0 ** -23) * mag)
    return out


def _check(nq, B, E, k, d, f, group, zeros, dtype, renormalise, seed=0):
    GU, gu, D, dn, X, R = _setup(B, E, d, f, group, zeros, dtype, seed)
    Y, ids, p = _run(nq, X, R, gu, dn, k, group, renormalise, want_routing=True)
    Xd = X.double().numpy()
    ry, rids, rp = O.moe(Xd, R.double().numpy(), GU, D, k, renormalise)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(p.cpu().numpy(), rp, rtol=2.0 ** -23, atol=0)
    assert (np.abs(Y.cpu().double().numpy() - ry) <= _y_bound(Xd, GU, D, rids, rp)).all()


@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,E,k,d,f", [(1, 1, 1, 1, 1), (1, 4, 2, 64, 32), (3, 5, 5, 33, 65),
                                       (2, 8, 3, 257, 40), (8, 16, 4, 160, 96), (16, 4, 2, 128, 130),
                                       (64, 3, 2, 96, 17), (64, 70, 16, 40, 24), (5, 512, 7, 48, 8)])
def test_moe_matches_the_oracle(nq, B, E, k, d, f, group, zeros, dtype):
    _check(nq, B, E, k, d, f, group, zeros, dtype, renormalise=B % 2 == 1, seed=B + E)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalise", [True, False])
def test_moe_at_a_larger_size(nq, dtype, renormalise):
    _check(nq, 12, 16, 4, 1000, 700, 128, True, dtype, renormalise, seed=3)
    _check(nq, 1, 32, 6, 2048, 512, 64, False, dtype, renormalise, seed=4)


def test_all_tokens_on_one_expert_and_equal_logits(nq):
    GU, gu, D, dn, X, R = _setup(40, 6, 64, 48, 32, True, torch.float32, 11)
    X[:, 0], R[:] = 3.0, 0.0
    R[4, 0] = 1.0                                   # expert 4 first, then 0 and 1 of a five-way tie
    Y, ids, p = _run(nq, X, R, gu, dn, 3, 32, True, want_routing=True)
    np.testing.assert_array_equal(ids.cpu().numpy(), np.tile([4, 0, 1], (40, 1)))
    ry, rids, rp = O.moe(X.double().numpy(), R.double().numpy(), GU, D, 3, True)
    assert (np.abs(Y.cpu().double().numpy() - ry) <= _y_bound(X.double().numpy(), GU, D, rids, rp)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_tokens_result_does_not_depend_on_the_others(nq, dtype):
    _, gu, _, dn, X, R = _setup(20, 8, 128, 96, 64, True, dtype, 13)
    Y, ids, p = _run(nq, X, R, gu, dn, 2, 64, True, want_routing=True)
    for b in (0, 7, 19):
        assert torch.equal(_run(nq, X[b:b + 1], R, gu, dn, 2, 64, True), Y[b:b + 1])
    bad = X.clone()
    bad[7, 3] = float("nan")
    out, bids, _ = _run(nq, bad, R, gu, dn, 2, 64, True, want_routing=True)
    keep = torch.arange(20) != 7
    assert torch.equal(out[keep.cuda()], Y[keep.cuda()]) and out[7].isnan().all()
    assert ((bids >= 0) & (bids < 8)).all()
    bad[7] = float("inf")
    out, bids, _ = _run(nq, bad, R, gu, dn, 2, 64, False, want_routing=True)
    assert torch.equal(out[keep.cuda()], _run(nq, X, R, gu, dn, 2, 64, False)[keep.cuda()])
    assert ((bids >= 0) & (bids < 8)).all()


def test_calls_in_graphs_that_share_a_workspace_and_on_two_streams(nq):
    _, gu, _, dn, X, R = _setup(6, 8, 256, 128, 64, False, torch.bfloat16, 17)
    ref = _run(nq, X, R, gu, dn, 2, 64, True)
    need = nq.lib.nq_moe_workspace_size(6, 256, 128, 8, 2, nq.NQ_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    static, Rc = X.cuda().clone(), R.cuda()
    graphs, outs = [], []
    for k in (2, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(nq.nq_moe_w4(static, Rc, gu[0], gu[1], dn[0], dn[1], k, group=64, ws=ws))
        graphs.append(g)
    one = _run(nq, X, R, gu, dn, 1, 64, True)
    for _ in range(3):
        for g, o, r in zip(graphs, outs, (ref, one)):
            g.replay()
            assert torch.equal(o, r)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(nq.nq_moe_w4(static, Rc, gu[0], gu[1], dn[0], dn[1], 2, group=64))
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in got)


def test_a_run_of_the_operators(nq):
    """Quantised experts behind a quantised projection, as a block would use them."""
    rng = np.random.default_rng(41)
    d, f, E, B = 128, 96, 4, 3
    dense = {k: 0.05 * torch.from_numpy(rng.standard_normal(s)).float().cuda()
             for k, s in (("proj", (d, d)), ("gu", (E * 2 * f, d)), ("dn", (E * d, f)))}
    q = {k: nq.nq_w4_quantize(w, group=32, symmetric=False, grid=4) for k, w in dense.items()}
    back = {k: nq.nq_w4_dequantize(v["packed"], v["scales"], dense[k].shape[1], 32, v["zeros"])
            .cpu().double().numpy() for k, v in q.items()}
    X = acts(B, d, torch.float32, 1)
    R = acts(E, d, torch.float32, 2)
    h = nq.nq_w4_matmul(q["proj"]["packed"], q["proj"]["scales"], X.cuda(), 32, q["proj"]["zeros"])
    st = lambda v, rows: tuple(v[n].view(E, rows, -1) for n in ("packed", "scales", "zeros"))  # noqa: E731
    Y = _run(nq, h, R, st(q["gu"], 2 * f), st(q["dn"], d), 2, 32, True)
    hd = h.cpu().double().numpy()
    GU, D = back["gu"].reshape(E, 2 * f, d), back["dn"].reshape(E, d, f)
    ry, ids, p = O.moe(hd, R.double().numpy(), GU, D, 2, True)
    assert (np.abs(Y.cpu().double().numpy() - ry) <= _y_bound(hd, GU, D, ids, p)).all()
    ref = O.matmul(X.double().numpy(), back["proj"])
    mag = O.matmul(np.abs(X.double().numpy()), np.abs(back["proj"]))
    assert (np.abs(hd - ref) <= product_bound(d) * mag).all()


def test_wrapper_refuses_what_does_not_fit(nq):
    _, gu, _, dn, X, R = _setup(2, 4, 64, 32, 32, False, torch.bfloat16, 1)
    X, R = X.cuda(), R.cuda()

    def call(X=X, R=R, gu=gu, dn=dn, k=2, group=32, **kw):
        return nq.nq_moe_w4(X, R, gu[0], gu[1], dn[0], dn[1], k, group=group, **kw)
    call()
    for bad in (dict(X=X[:, :32]), dict(R=R[:3]), dict(R=R.float()), dict(group=64), dict(group=5),
                dict(gu=dn), dict(dn=gu), dict(X=X[0]), dict(gu=(gu[0][0], gu[1][0]))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(k=0), dict(k=5), dict(X=torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(nq.NQError):
            call(**bad)
