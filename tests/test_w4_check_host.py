"""Host-side checks of the 4-bit calls' status entry points (CPU only: no device is touched)."""
import pytest
import torch

import rank_binary_factorization_b200 as nq

L = nq.lib
OK, INV, WS = nq._lib.NQ_OK, nq._lib.NQ_ERR_INVALID_ARG, nq._lib.NQ_ERR_WORKSPACE
FAKE = 1 << 40


def test_matmul_check_refuses():
    def call(m=64, n=4096, dt=0, B=99, ws=FAKE, ws_bytes=1 << 30):
        return L.nq_w4_check(m, n, dt, B, ws, ws_bytes, None)
    for bad in (dict(m=0), dict(n=0), dict(n=65537), dict(dt=2), dict(B=0), dict(B=65537), dict(ws=None),
                dict(ws=FAKE + 64)):
        assert call(**bad) == INV, bad
    assert call(ws_bytes=64) == WS
    # calls without waits: no workspace, or one for the columns alone
    assert call(n=64, B=1, ws=None, ws_bytes=0) == OK
    assert call(n=65536, B=2) == OK


def test_moe_check_refuses():
    def call(B=2, d=64, f=32, E=4, top_k=2, dt=1, ws=FAKE, ws_bytes=1 << 30):
        return L.nq_moe_check(B, d, f, E, top_k, dt, ws, ws_bytes, None)
    for bad in (dict(B=0), dict(B=65), dict(d=0), dict(f=0), dict(E=0), dict(top_k=5), dict(dt=2),
                dict(ws=None), dict(ws=FAKE + 8)):
        assert call(**bad) == INV, bad
    assert call(ws_bytes=64) == WS


def test_wrappers_refuse_a_workspace_on_the_host():
    ws = torch.empty(1024, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nq.nq_w4_check(64, 64, torch.float32, 99, ws)
    with pytest.raises(ValueError):
        nq.nq_moe_check(1, 64, 32, 4, 2, torch.float32, ws)


def test_wrappers_refuse_other_types():
    ws = torch.empty(1024, dtype=torch.uint8)
    with pytest.raises(TypeError):
        nq.nq_w4_check(64, 64, torch.float16, 99, ws)
    with pytest.raises(TypeError):
        nq.nq_moe_check(1, 64, 32, 4, 2, torch.int8, ws)
