"""Sizes that one launch cannot hold, refused on the host (no GPU: nothing
here launches a kernel, and no pointer is dereferenced)."""
import pytest

from test_mixer_boundary import INVALID, OK, UNSUPPORTED, P, conv_bwd, conv_fwd, conv_step, norm_bwd, norm_fwd


@pytest.mark.parametrize("bad", [
    dict(T=1 << 30, D=64), dict(T=(1 << 31) - 300, D=1, xs=1), dict(T=1 << 20, N=1 << 30, cu=P, out=P),
    dict(T=(1 << 31) - 300, N=(1 << 31) - 1, cu=P, out=P, D=1, xs=1),
])
def test_conv_fwd_more_tokens_than_threads(bad):
    assert conv_fwd(**bad) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(D=(1 << 24) - 1, xs=1 << 24, dys=1 << 24, nbytes=1 << 40)])
def test_conv_bwd_more_channels_than_blocks(bad):
    assert conv_bwd(**bad) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(R=1 << 26, Pn=1 << 26), dict(R=(1 << 31) - 1, Pn=4), dict(D=(1 << 24) - 1, xs=1 << 24),
])
def test_conv_step_more_requests_than_threads(bad):
    assert conv_step(**bad) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(R=1 << 28, D=64), dict(R=1 << 28, D=7), dict(R=1 << 22, D=8192), dict(R=1 << 22, D=8191), dict(R=1 << 27, D=128, dt=0),
])
def test_norm_fwd_more_rows_than_threads(bad):
    assert norm_fwd(**bad) == UNSUPPORTED


@pytest.mark.parametrize("gate,G,want", [(P, 0, OK), (P, 1, OK), (P, 5, OK), (None, 0, OK), (P, -1, INVALID)])
def test_norm_without_rows(gate, G, want):
    """No rows, and a gate of none (per row) or of any number (shared)."""
    assert norm_fwd(gate=gate, G=G, R=0) == want


@pytest.mark.parametrize("bad,want", [
    (dict(gate=P, dgate=None, G=1, R=0), INVALID), (dict(gate=P, dgate=P, G=-1, R=0), INVALID),
    (dict(gate=P, dgate=P, G=0, R=4), INVALID), (dict(gate=None, dgate=P, G=4, R=0), INVALID),
])
def test_norm_bwd_gates_without_rows(bad, want):
    assert norm_bwd(**bad) == want
