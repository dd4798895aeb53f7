"""Host-side checks of the 4-bit entry points (CPU only: no kernel is launched)."""
import ctypes

import pytest
import torch

import rank_binary_factorization_b200 as nq

L = nq.lib
INV, WS = nq._lib.NQ_ERR_INVALID_ARG, nq._lib.NQ_ERR_WORKSPACE
FAKE = 1 << 40     # never dereferenced: every call below fails validation first


def _quantize(W=FAKE, dt=1, m=8, n=64, d_in=None, group=32, grid=1, packed=FAKE, scales=FAKE):
    return L.nq_w4_quantize(W, dt, m, n, d_in, group, grid, packed, scales, None, None)


def test_quantize_refuses():
    for bad in (dict(W=None), dict(dt=2), dict(m=0), dict(m=(1 << 24) + 1), dict(n=0), dict(n=65537),
                dict(group=16), dict(group=256), dict(grid=0), dict(grid=65), dict(packed=None),
                dict(packed=FAKE + 4), dict(scales=None), dict(scales=FAKE + 1), dict(W=FAKE + 1),
                dict(d_in=FAKE + 2), dict(dt=0, W=FAKE + 2)):
        assert _quantize(**bad) == INV, bad


def test_dequantize_refuses():
    def call(packed=FAKE, scales=FAKE, m=8, n=64, group=32, W=FAKE, dt=0):
        return L.nq_w4_dequantize(packed, scales, None, m, n, group, W, dt, None)
    for bad in (dict(packed=None), dict(scales=None), dict(m=-1), dict(n=0), dict(group=48),
                dict(W=None), dict(W=FAKE + 2), dict(dt=5)):
        assert call(**bad) == INV, bad


def test_matmul_refuses():
    def call(packed=FAKE, scales=FAKE, m=8, n=64, group=32, X=FAKE, dt=0, B=99, Y=FAKE, ws=FAKE,
             ws_bytes=1 << 30):
        return L.nq_w4_matmul(packed, scales, None, m, n, group, X, dt, B, Y, ws, ws_bytes, None)
    for bad in (dict(packed=None), dict(packed=FAKE + 8), dict(scales=None), dict(m=0), dict(n=0),
                dict(group=0), dict(X=None), dict(X=FAKE + 2), dict(dt=3), dict(B=0),
                dict(B=65537), dict(Y=None), dict(Y=FAKE + 1), dict(ws=None), dict(ws=FAKE + 64)):
        assert call(**bad) == INV, bad
    assert call(ws_bytes=16) == WS


def test_moe_refuses():
    def call(X=FAKE, dt=1, B=2, d=64, router=FAKE, E=4, top_k=2, renorm=1, gu=FAKE, gus=FAKE, dn=FAKE,
             dns=FAKE, f=32, group=32, Y=FAKE, ids=None, weights=None, ws=FAKE, ws_bytes=1 << 30):
        return L.nq_moe_w4(X, dt, B, d, router, E, top_k, renorm, gu, gus, None, dn, dns, None, f, group,
                           Y, ids, weights, ws, ws_bytes, None)
    for bad in (dict(X=None), dict(dt=4), dict(B=0), dict(B=65), dict(d=0), dict(router=None), dict(E=0),
                dict(E=513), dict(top_k=0), dict(top_k=5), dict(E=40, top_k=17), dict(renorm=2),
                dict(gu=None), dict(gu=FAKE + 4), dict(gus=None), dict(dn=None), dict(dns=None),
                dict(f=0), dict(group=100), dict(Y=None), dict(ids=FAKE + 2), dict(weights=FAKE + 1),
                dict(ws=None), dict(ws=FAKE + 8), dict(E=512, f=32768, top_k=1)):
        assert call(**bad) == INV, bad
    assert call(ws_bytes=64) == WS


def test_workspace_sizes():
    assert L.nq_w4_workspace_size(64, 64, 0, 99) > 0
    assert L.nq_w4_workspace_size(64, 64, 0, 0) == 0
    assert L.nq_w4_workspace_size(0, 64, 0, 1) == 0
    small, large = (L.nq_moe_workspace_size(b, 64, 32, 4, 2, 0) for b in (1, 64))
    assert 0 < small < large
    assert L.nq_moe_workspace_size(65, 64, 32, 4, 2, 0) == 0
    assert L.nq_moe_workspace_size(1, 64, 32, 4, 5, 0) == 0


def test_python_wrappers_refuse_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(2, 64)
    packed, scales = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nq.nq_w4_quantize(x, group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_dequantize(packed, scales, 64, group=32)
    with pytest.raises(ValueError):
        nq.nq_w4_matmul(packed, scales, x, group=32)
    with pytest.raises(ValueError):
        nq.nq_moe_w4(x, x, packed[None], scales[None], packed[None], scales[None], 1, group=32)
