"""Host-side checks of the setting of the 4-bit products' waits (CPU only)."""
import pytest

import rank_binary_factorization_b200 as nq


def test_wait_polls_are_checked():
    for v in (0, 1, 1 << 30, -1):
        assert nq.lib.nq_set_w4_wait_polls(v) == nq._lib.NQ_OK
    assert nq.lib.nq_set_w4_wait_polls(-2) == nq._lib.NQ_ERR_INVALID_ARG
    with pytest.raises(nq.NQError):
        nq.nq_set_w4_wait_polls(-7)
    nq.nq_set_w4_wait_polls()
