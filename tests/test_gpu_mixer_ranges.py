"""The sequence-mixing operators where magnitudes, decays and counts lie far
apart, against their 64-bit definitions: cleared states, tokens and heads
that dwarf their neighbours, many sequences and many heads of one key.

Tolerances are those of test_gpu_mixer.py: half a step of the result's type,
and 1e-5 of its norm for a forward pass of the delta rule, 2e-5 for a forward
and a backward one.  They are asked of each part of a result by itself (a
chunk, a head), not of the whole, whose norm a large part would decide.
"""
import pytest
import torch

from convolution_lowering_amd import mixer
from oracle import mixer as om
from test_gpu_mixer import DEV, T16, _cu, _delta_inputs, _delta_ref, _gen, _near, _randn, _say

pytestmark = pytest.mark.gpu


# ------------------------------------------- gated delta rule: cleared states


def _parts(got, ref, what, loose=1e-5):
    """Chunks of 64 tokens, each by its own norm."""
    for t in range(0, ref.shape[0], 64):
        _near(got[t:t + 64], ref[t:t + 64], f"{what}[{t}:]", loose)


def _clears(kind, dtype):
    """200 tokens whose first chunk, or second, wipes out what was large and
    adds nothing; the tokens after it are ordinary."""
    q, k, v, g, beta, gen = _delta_inputs([200], 1, 2, 64, 64, dtype, packed=False, fast=0.1)
    state = None
    if kind == "state":      # a large state cleared by a chunk that writes nothing
        state = 4e4 * _randn(gen, 1, 2, 64, 64)
        g[0] = -float("inf")
        beta[:64] = 0
    elif kind == "values":   # large values, then a cleared chunk without values
        v[:64] *= 3e4
        g[64] = -float("inf")
        v[64:128] = 0
    elif kind == "inside":   # the clear lies inside a chunk that writes nothing
        v[:64] *= 3e4
        g[100] = -float("inf")
        beta[64:128] = 0
    elif kind == "no key":   # a large value under a key of zeros, then no values: no clear at all
        v[:128] = 0
        v[1], k[1] = 1e7, 0
    else:                    # nothing is written of huge values
        v[:64] *= 1e9
        beta[:64] = 0
    return q, k, v, g, beta, state


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["state", "values", "inside", "no key", "unwritten"])
def test_delta_rule_chunks_that_clear_and_add_nothing(kind, dtype):
    _say("delta clears", kind, dtype)
    q, k, v, g, beta, state = _clears(kind, dtype)
    o, s, _ = mixer.delta_rule_fwd(q, k, v, g, beta, state=state, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(q, k, v, g, beta, None, state, 0.125, True)
    _parts(o, ro, "o")
    _near(s, rs, "state")


@pytest.mark.parametrize("what", ["beta", "v"])
def test_delta_rule_one_token_clears_a_large_state(what):
    q, k, v, g, beta, gen = _delta_inputs([1], 1, 1, 64, 64, "bf16", packed=False)
    (beta if what == "beta" else v).zero_()
    g.fill_(-float("inf"))
    state = 4e4 * _randn(gen, 1, 1, 64, 64)
    o, s, _ = mixer.delta_rule_fwd(q, k, v, g, beta, state=state, qk_norm=True, want_state=True)
    assert (o == 0).all() and (s == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["clear", "unwritten"])
def test_delta_rule_gradients_of_a_cleared_chunk(kind, dtype):
    """The second chunk clears the state at its first token (or last, and
    writes nothing) and has no output gradient; the gradients after it are
    large, as a scaled loss makes them."""
    _say("delta clears, gradients", kind, dtype)
    q, k, v, g, beta, gen = _delta_inputs([200], 1, 2, 64, 64, dtype, packed=False, fast=0.1)
    g[64 if kind == "clear" else 127] = -5000.0  # zero in 64 bits as well
    if kind == "unwritten":
        beta[64:128] = 0
    state = _randn(gen, 1, 2, 64, 64)
    do = (1e7 * _randn(gen, 200, 2, 64)).to(v.dtype)
    do[64:128] = 0
    ds = 1e7 * _randn(gen, 1, 2, 64, 64)
    more = dict(scale=0.125, qk_norm=True)
    _, _, saved = mixer.delta_rule_fwd(q, k, v, g, beta, state=state, save=True, **more)
    got = mixer.delta_rule_bwd(do, q, k, v, g, beta, saved, dstate_out=ds, want_dstate=True, **more)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, g, beta, state)]
    ro, rs = om.delta_rule(*leaves[:5], None, leaves[5], 0.125, True)
    ref = torch.autograd.grad((ro * do.double()).sum() + (rs * ds.double()).sum(), leaves)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), got, ref):
        _near(x, y, name, 2e-5)
