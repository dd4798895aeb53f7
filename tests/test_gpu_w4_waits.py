"""Device-side waits of the 4-bit products that run out: the call ends, and what they kept from being
computed is NaN.

The waits are given so few polls that they run out in a healthy call.  How far a call gets is then
chance, but an element is either NaN or the bits of the undisturbed call, and the next call is whole.
"""
import pytest
import torch

from w4_common import acts, layer, stack

pytestmark = pytest.mark.gpu


@pytest.fixture
def polls(nq):
    yield nq.nq_set_w4_wait_polls
    nq.nq_set_w4_wait_polls()


def _nan_or_same(Y, ref):
    assert (Y.isnan() | (Y == ref)).all()


# tiles of 32, 64 and 128 columns, one or three terms, all groups; one unit a CTA, several, split axes
CASES = [(6000, 1100, 513, torch.bfloat16, 128, False), (20000, 1100, 50, torch.bfloat16, 64, True),
         (25600, 1100, 20, torch.float32, 32, True), (2000, 1100, 300, torch.float32, 128, True),
         (40, 65536, 24, torch.bfloat16, 32, False), (300, 2000, 100, torch.float32, 64, False),
         (1, 1, 17, torch.bfloat16, 128, True)]


@pytest.mark.parametrize("m,n,B,dtype,group,zeros", CASES)
def test_products_whose_waits_run_out(nq, polls, m, n, B, dtype, group, zeros):
    _, (packed, scales, z) = layer(m, n, group, zeros, m)
    X = acts(B, n, dtype, 1).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=group, zeros=z)
    assert ref.isfinite().all()
    polls(0)
    assert nq.nq_w4_matmul(packed, scales, X, group=group, zeros=z).isnan().all()
    for limit in (1, 2, 5, 20, 100, 1000):
        polls(limit)
        for _ in range(3):
            _nan_or_same(nq.nq_w4_matmul(packed, scales, X, group=group, zeros=z), ref)
    polls()
    assert torch.equal(nq.nq_w4_matmul(packed, scales, X, group=group, zeros=z), ref)


def test_calls_without_waits_are_not_touched(nq, polls):
    _, (packed, scales, z) = layer(300, 2000, 64, True, 3)
    X = acts(4, 2000, torch.float32, 4).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z)
    polls(0)
    assert torch.equal(nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z), ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 20])
def test_expert_layers_whose_waits_run_out(nq, polls, B, dtype):
    _, gu = stack(6, 2 * 700, 1000, 64, True, 5)
    _, dn = stack(6, 1000, 700, 64, True, 6)
    X, R = acts(B, 1000, dtype, 7).cuda(), acts(6, 1000, dtype, 8).cuda()

    def call():
        return nq.nq_moe_w4(X, R, gu[0], gu[1], dn[0], dn[1], 2, group=64, gate_up_zeros=gu[2],
                            down_zeros=dn[2])
    ref = call()
    assert ref.isfinite().all()
    for limit in (0, 1, 10, 100):
        polls(limit)
        for _ in range(3):
            Y = call()
            _nan_or_same(Y, ref)
            assert limit > 0 or Y.isnan().any()
    polls()
    assert torch.equal(call(), ref)


def test_waits_that_run_out_on_two_streams(nq, polls):
    _, (packed, scales, z) = layer(6000, 1100, 64, True, 9)
    X = acts(100, 1100, torch.bfloat16, 10).cuda()
    ref = nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for limit in (3, -1, 0, -1):
        polls(limit)
        for s in streams:
            with torch.cuda.stream(s):
                out.append((limit, nq.nq_w4_matmul(packed, scales, X, group=64, zeros=z)))
    torch.cuda.synchronize()
    for limit, Y in out:
        assert torch.equal(Y, ref) if limit < 0 else Y.isnan().all() if limit == 0 else True
        _nan_or_same(Y, ref)
