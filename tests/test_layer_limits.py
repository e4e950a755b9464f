"""Calls beyond a launch's limits are refused on the host, before anything is enqueued."""
import pytest

import w4a16_group_wise_amd as w4q

A = 4096  # a fake address, never dereferenced: the checks fail first


# the fake-quantised write takes 8 weights a thread, and a launch counts its threads below 2^32
@pytest.mark.parametrize("d_out,d_in", [(1 << 29, 128), (1 << 21, 1 << 14), ((1 << 28) - 1, 128), (1 << 25, 1024)])
def test_weights_past_one_launch_are_refused(d_out, d_in):
    got = w4q.lib().lsq_linear_fwd(A, 1, A, A, d_out, d_in, None, 0, None, A, None, A, 1, None, 0, None)
    assert got == w4q.W4Q_EUNSUPPORTED


def test_steps_are_whole_numbers_that_fit():
    from w4a16_group_wise_amd import ops

    assert ops._steps(5) == 5 and ops._steps(5.0) == 5 and ops._steps(0) == 0
    for bad in (2.5, 2 ** 32 + 5, -2 ** 31 - 1, float("inf"), float("nan")):
        with pytest.raises((ValueError, OverflowError)):
            ops._steps(bad)
