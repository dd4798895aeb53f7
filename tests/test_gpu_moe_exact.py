"""Expert layer on long axes, where every sum is exact in FP32.

Gates are whole numbers above 18, where 1 + exp(-g) rounds to 1 and silu(g) to g; one expert a token
has the weight 1; so y = D ((G x) * (U x)) in whole numbers.
"""
import numpy as np
import pytest
import torch

from oracle import w4 as O
from w4_exact import assert_exact, to_gpu

pytestmark = pytest.mark.gpu


def _sparse(rng, shape, share, low, high):
    """Whole numbers low .. high in a share of the places, 0 elsewhere."""
    return np.where(rng.random(shape) < share, rng.integers(low, high + 1, shape, dtype=np.int8), 0).astype(np.int8)


def _inputs(E, d, f, B, group, zeros, seed):
    rng = np.random.default_rng(seed)
    # code - zero point: gates with one large first column, dense up rows, sparse down rows
    gate = _sparse(rng, (E * f, d), 0.1, -1, 1)
    gate[:, 0] = rng.integers(5, 8, E * f)
    up = rng.integers(-7, 8, (E * f, d), dtype=np.int8)
    gu = np.concatenate([gate.reshape(E, f, d), up.reshape(E, f, d)], 1)
    dn = _sparse(rng, (E, d, f), min(1.0, 30 / f), -7, 7)
    stacks = []
    for a in (gu, dn):
        rows, n = a.shape[0] * a.shape[1], a.shape[2]
        z = np.full((rows, -(-n // group)), 7) if zeros else None
        t = to_gpu(a.reshape(rows, n) + (7 if zeros else 8), np.ones((rows, -(-n // group))), z)
        stacks.append(tuple(None if v is None else v.view(E, a.shape[1], -1) for v in t))
    # activations in places that differ from token to token
    X = _sparse(rng, (B, d), min(1.0, 12 / d), -3, 3).astype(np.float64)
    X[:, 0] = 16
    R = torch.from_numpy(rng.standard_normal((E, d)) * (np.arange(d) != 0)).float()
    R[:, 0] = 0.001 * torch.randperm(E)       # tokens whose places meet none of a router row
    return gu.astype(np.float64), dn.astype(np.float64), *stacks, X, R


@pytest.mark.parametrize("d,f", [(4173, 4200), (300, 8500), (8500, 300), (4096, 129), (65536, 40),
                                 (64, 65536)])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_on_long_axes(nq, d, f, dtype, group, zeros):
    E = 2
    GU, D, gu, dn, X, R = _inputs(E, d, f, 23, group, zeros, d + group)
    R = R.to(dtype)
    ids, p = O.route(X, R.double().numpy(), 1, True)
    ref = np.zeros_like(X)
    for b, e in enumerate(ids[:, 0]):
        g, u = GU[e, :f] @ X[b], GU[e, f:] @ X[b]
        assert (g > 18).all()
        h = g * u
        assert_exact(h[None], D[e], 1)
        ref[b] = D[e] @ h
    need = nq.lib.nq_moe_workspace_size(23, d, f, E, 1, nq.NQ_BF16 if dtype == torch.bfloat16 else nq.NQ_F32)
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    for B in (1, 4, 23):
        Y, got, w = nq.nq_moe_w4(torch.from_numpy(X[:B]).to(dtype).cuda(), R.cuda(), gu[0], gu[1], dn[0],
                                 dn[1], 1, group=group, gate_up_zeros=gu[2], down_zeros=dn[2],
                                 want_routing=True, ws=ws[:need])
        np.testing.assert_array_equal(got.cpu().numpy(), ids[:B])
        assert (w == 1).all()
        np.testing.assert_array_equal(Y.cpu().double().numpy(), ref[:B])
        assert (ws[need:] == 171).all()
