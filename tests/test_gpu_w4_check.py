"""The status word of the 4-bit calls: raised by a wait that ran out, cleared by the next call."""
import pytest
import torch

from w4_common import acts, layer, stack

pytestmark = pytest.mark.gpu


@pytest.fixture
def polls(nq):
    yield nq.nq_set_w4_wait_polls
    nq.nq_set_w4_wait_polls()


# one part of the k axis, several, and FP32 terms; the word lies behind the parts
@pytest.mark.parametrize("m,n,B,dtype", [(6000, 300, 500, torch.bfloat16), (65, 8192, 20, torch.float32),
                                         (33, 1025, 17, torch.bfloat16)])
def test_matmul_reports_a_wait_that_ran_out(nq, polls, m, n, B, dtype):
    _, (packed, scales, z) = layer(m, n, 64, True, 1)
    X = acts(B, n, dtype, 2).cuda()
    need = nq.lib.nq_w4_workspace_size(m, n, nq.NQ_BF16 if dtype == torch.bfloat16 else nq.NQ_F32, B)
    whole = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    ws = whole[:need]

    def call():
        Y = nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z, ws=ws)
        return Y, nq.nq_w4_check(m, n, dtype, B, ws)
    ref, code = call()
    assert code == 0 and ref.isfinite().all()
    polls(0)
    Y, code = call()
    assert code == nq._lib.NQ_ERR_TIMEOUT and Y.isnan().all()
    polls()
    Y, code = call()
    assert code == 0 and torch.equal(Y, ref)
    assert (whole[need:] == 255).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_report_a_wait_that_ran_out(nq, polls, dtype):
    B, d, f, E, k = 5, 200, 130, 6, 2
    _, gu = stack(E, 2 * f, d, 32, False, 5)
    _, dn = stack(E, d, f, 32, False, 6)
    X, R = acts(B, d, dtype, 7).cuda(), acts(E, d, dtype, 8).cuda()
    need = nq.lib.nq_moe_workspace_size(B, d, f, E, k, nq.NQ_BF16 if dtype == torch.bfloat16 else nq.NQ_F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")

    def call():
        Y = nq.nq_moe_w4(X, R, gu[0], gu[1], dn[0], dn[1], k, group=32, ws=ws)
        return Y, nq.nq_moe_check(B, d, f, E, k, dtype, ws)
    ref, code = call()
    assert code == 0 and ref.isfinite().all()
    polls(0)
    Y, code = call()
    assert code == nq._lib.NQ_ERR_TIMEOUT and Y.isnan().any()
    polls()
    Y, code = call()
    assert code == 0 and torch.equal(Y, ref)


def test_a_nan_weight_is_not_reported(nq):
    m, n, B = 200, 512, 40
    _, (packed, scales, _) = layer(m, n, 128, False, 3)
    scales[5, 1] = float("nan")
    ws = nq.workspace(nq.lib.nq_w4_workspace_size(m, n, nq.NQ_BF16, B))
    Y = nq.nq_w4_matmul(packed, scales, acts(B, n, torch.bfloat16, 4).cuda(), group=128, ws=ws)
    assert Y[:, 5].isnan().all() and nq.nq_w4_check(m, n, torch.bfloat16, B, ws) == 0


def test_a_captured_call_reports_at_every_replay(nq, polls):
    m, n, B = 300, 1000, 60
    _, (packed, scales, z) = layer(m, n, 32, True, 9)
    X = acts(B, n, torch.bfloat16, 10).cuda()
    ws = nq.workspace(nq.lib.nq_w4_workspace_size(m, n, nq.NQ_BF16, B))
    ref = nq.nq_w4_matmul(packed, scales, X, group=32, zeros=z, ws=ws)
    graphs = []
    for limit in (0, -1):
        polls(limit)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = nq.nq_w4_matmul(packed, scales, X, group=32, zeros=z, ws=ws)
        graphs.append((g, Y))
    for _ in range(2):
        graphs[0][0].replay()
        assert nq.nq_w4_check(m, n, torch.bfloat16, B, ws) == nq._lib.NQ_ERR_TIMEOUT
        graphs[1][0].replay()
        assert nq.nq_w4_check(m, n, torch.bfloat16, B, ws) == 0 and torch.equal(graphs[1][1], ref)
