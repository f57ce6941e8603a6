"""Calls of the feed-forward operators that are refused after their sizes are
found to be too large for one launch: nothing is launched first (no GPU: a launch
would give another status)."""
import pytest

from test_ffn_boundary import P, UNSUPPORTED, bwd


@pytest.mark.parametrize("size", [
    dict(T=(1 << 31) - 300, D=1 << 10, xs=1 << 10, F=1),  # dx: 2^25 x 2^4 blocks of 256 threads
    dict(T=8, D=1 << 20, xs=1 << 20, F=1 << 20, dhs=1 << 20),  # dw_gate and dw_up: 2^13 x 2^12 of 512
], ids=["dx", "dw"])
def test_gradients_that_no_launch_holds(size):
    assert bwd(**size, sb=1 << 62, nbytes=1 << 62, ws=P, saved=P) == UNSUPPORTED
