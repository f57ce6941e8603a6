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


# ------------------------------------- gated delta rule: parts far from others


def _room(large, ordinary):
    """What an operand's split leaves out of a value that much smaller than
    its column's largest: half of f16's smallest step, where the largest is at
    2^11 or above; for two operands in series."""
    return 2 * 2.0 ** -36 * large / ordinary


@pytest.mark.parametrize("times", [1e2, 1e5])
def test_delta_rule_a_large_value_that_decays(times):
    """One token of a chunk holds values far above the others'; it has decayed
    to nothing before the chunk ends.  The state after it is made of ordinary
    tokens and keeps its digits."""
    _say("delta, one large value", times)
    q, k, v, g, beta, gen = _delta_inputs([256], 1, 2, 64, 64, "fp32", packed=False)
    v = _randn(gen, 256, 2, 64)
    g.fill_(-0.5)
    v[2] *= times
    v[130] *= times
    o, s, _ = mixer.delta_rule_fwd(q, k, v, g, beta, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(q, k, v, g, beta, None, None, 0.125, True)
    loose = 1e-5 + _room(v.abs().max().item(), 1.0)
    for t in range(0, 256, 16):
        _near(o[t:t + 16], ro[t:t + 16], f"o[{t}:]", loose)
    _near(s, rs, "state", loose)
    o, s, _ = mixer.delta_rule_fwd(*(z[:64].contiguous() for z in (q, k, v, g, beta)), qk_norm=True, want_state=True)
    _near(s, _delta_ref(*(z[:64] for z in (q, k, v, g, beta)), None, None, 0.125, True)[1], "state of a chunk", loose)


@pytest.mark.parametrize("times", [1e2, 1e5])
def test_delta_rule_a_large_output_gradient_that_decays(times):
    _say("delta, one large output gradient", times)
    q, k, v, g, beta, gen = _delta_inputs([192], 1, 2, 64, 64, "fp32", packed=False)
    g.fill_(-0.5)
    do = _randn(gen, 192, 2, 64)
    do[125] *= times
    state = _randn(gen, 1, 2, 64, 64)
    more = dict(scale=0.125, qk_norm=True)
    _, _, saved = mixer.delta_rule_fwd(q, k, v, g, beta, state=state, save=True, **more)
    got = mixer.delta_rule_bwd(do, q, k, v, g, beta, saved, want_dstate=True, **more)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, g, beta, state)]
    ro, _ = om.delta_rule(*leaves[:5], None, leaves[5], 0.125, True)
    ref = torch.autograd.grad((ro * do.double()).sum(), leaves)
    loose = 2e-5 + 2 * _room(do.abs().max().item(), 1.0)
    for t in range(0, 192, 16):
        _near(got[2][t:t + 16], ref[2][t:t + 16], f"dv[{t}:]", loose)
    _near(got[5], ref[5], "dstate", loose)


def _shared(dtype, heads=4, tokens=150):
    q, k, v, g, beta, gen = _delta_inputs([tokens], 1, heads, 64, 64, dtype, packed=False, beta32=True)
    return q, k, v, g, beta, _randn(gen, tokens, heads, 64), gen


def _bwd(do, *five):
    more = dict(scale=0.125, qk_norm=True)
    _, _, saved = mixer.delta_rule_fwd(*five, save=True, **more)
    return mixer.delta_rule_bwd(do, *five, saved, **more)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scales", [(1.0, 1e4, 1.0, 1e-2), (1e5, 1e-3, 1e-3, 1.0)])
def test_delta_rule_gradients_of_heads_of_different_size(scales, dtype):
    """Value heads that share a key: each one's decay and beta gradients keep
    the digits of its own size."""
    _say("delta, heads of different size", scales, dtype)
    q, k, v, g, beta, do, _ = _shared(dtype)
    do = (do * torch.tensor(scales, device=DEV)[None, :, None]).to(v.dtype)
    got = _bwd(do, q, k, v, g, beta)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, g, beta)]
    ro, _ = om.delta_rule(*leaves, None, None, 0.125, True)
    ref = torch.autograd.grad(ro, leaves, do.double())
    for h in range(len(scales)):
        for i, name in ((2, "dv"), (3, "dg"), (4, "dbeta")):
            _near(got[i][:, h], ref[i][:, h], f"{name} of head {h}", 2e-5)
    for i, name in ((0, "dq"), (1, "dk")):
        _near(got[i], ref[i], name, 2e-5)


def test_delta_rule_a_broken_head_leaves_the_others():
    """One head's output gradient is NaN: the other heads' own gradients are
    those of a call without it."""
    q, k, v, g, beta, do, _ = _shared("bf16")
    whole = do.to(v.dtype)
    broken = whole.clone()
    broken[:, 1] = float("nan")
    a, b = _bwd(whole, q, k, v, g, beta), _bwd(broken, q, k, v, g, beta)
    for h in (0, 2, 3):
        for i, name in ((2, "dv"), (3, "dg"), (4, "dbeta")):
            assert torch.equal(a[i][:, h], b[i][:, h]), f"{name} of head {h}"
    assert b[3][:, 1].isnan().any()


# ------------------------------------------- gated delta rule: counts and zeros


@pytest.mark.parametrize("rep,dk,dv,dtype", [(6, 128, 128, "bf16"), (9, 40, 72, "fp32"), (5, 64, 64, "fp16")])
def test_delta_rule_many_value_heads_of_one_key(rep, dk, dv, dtype):
    _say("delta, value heads of one key", rep, dk, dv, dtype)
    q, k, v, g, beta, gen = _delta_inputs([70, 9], 2, 2 * rep, dk, dv, dtype)
    cu = _cu([70, 9])
    do = _randn(gen, 79, 2 * rep, dv).to(v.dtype)
    more = dict(cu_seqlens=cu, scale=0.2, qk_norm=True)
    o, s, saved = mixer.delta_rule_fwd(q, k, v, g, beta, want_state=True, save=True, **more)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, g, beta)]
    ro, rs = om.delta_rule(*leaves, cu.tolist(), None, 0.2, True)
    ref = torch.autograd.grad(ro, leaves, do.double())
    got = mixer.delta_rule_bwd(do, q, k, v, g, beta, saved, **more)
    _near(s, rs.detach(), "state")
    for h in range(2 * rep):
        _near(o[:, h], ro[:, h].detach(), f"o of head {h}")
        for i, name in ((2, "dv"), (3, "dg"), (4, "dbeta")):
            _near(got[i][:, h], ref[i][:, h], f"{name} of head {h}", 2e-5)
    for i, name in ((0, "dq"), (1, "dk")):
        _near(got[i], ref[i], name, 2e-5)


@pytest.mark.parametrize("n", [65, 200, 4100])
def test_delta_rule_many_sequences(n):
    """More sequences than a wavefront looks at together, some of them empty;
    each gives what it gives alone."""
    _say("delta, sequences", n)
    pick = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 4, (n,), generator=pick).tolist()
    for i, ln in ((3, 70), (64, 1), (n - 1, 130)):
        lens[i] = ln
    q, k, v, g, beta, gen = _delta_inputs(lens, 1, 1, 32, 32, "bf16", packed=False)
    state = _randn(gen, n, 1, 32, 32)
    cu = _cu(lens)
    at = cu.tolist()
    o, s, saved = mixer.delta_rule_fwd(q, k, v, g, beta, cu_seqlens=cu, state=state, qk_norm=True, want_state=True,
                                       save=True)
    do = _randn(gen, *v.shape).to(v.dtype)
    got = mixer.delta_rule_bwd(do, q, k, v, g, beta, saved, cu_seqlens=cu, qk_norm=True, want_dstate=True)
    some = [0, 1, 2, 3, 62, 63, 64, n // 2, n - 2, n - 1]
    for i in some:
        a, e = at[i], at[i + 1]
        if a == e:
            assert torch.equal(s[i], state[i]) and (got[5][i] == 0).all()
            continue
        five = [z[a:e].contiguous() for z in (q, k, v, g, beta)]
        o1, s1, saved1 = mixer.delta_rule_fwd(*five, state=state[i:i + 1], qk_norm=True, want_state=True, save=True)
        assert torch.equal(o[a:e], o1) and torch.equal(s[i:i + 1], s1), f"sequence {i}"
        g1 = mixer.delta_rule_bwd(do[a:e].contiguous(), *five, saved1, qk_norm=True, want_dstate=True)
        for x, y in zip(got[:5], g1[:5]):
            assert torch.equal(x[a:e], y), f"gradients of sequence {i}"
        assert torch.equal(got[5][i:i + 1], g1[5])
        ro, rs = _delta_ref(*five, None, state[i:i + 1], 32 ** -0.5, True)
        _near(o1, ro, f"sequence {i}")
        _near(s1, rs, f"state {i}")


@pytest.mark.parametrize("form", ["chunks", "tokens"])
def test_delta_rule_tokens_that_write_nothing(form):
    """beta = 0 for some tokens, or all: the state only decays there."""
    q, k, v, g, beta, gen = _delta_inputs([96], 1, 2, 64, 48, "bf16", packed=False)
    beta[torch.rand(96, 2, generator=gen, device=DEV) < 0.5] = 0
    beta[:, 1] = 0
    state = _randn(gen, 1, 2, 64, 48)
    ro, rs = _delta_ref(q, k, v, g, beta, None, state, 0.125, True)
    if form == "chunks":
        o, s, _ = mixer.delta_rule_fwd(q, k, v, g, beta, state=state, qk_norm=True, want_state=True)
    else:
        s = state.clone()
        o = mixer.delta_rule_step(q[None], k[None], v[None], g[None], beta[None], s, scale=0.125, qk_norm=True)[0]
    for h in range(2):
        _near(o[:, h], ro[:, h], f"o of head {h}")
        _near(s[:, h], rs[:, h], f"state of head {h}")


# ----------------------------------------------------- float32 results' digits


def _steps(got, ref):
    """Largest distance in half steps of float32, of the results that are
    not below its normal range."""
    there = ref.abs() > 2.0 ** -126
    return ((got.double() - ref).abs() / ref.abs())[there].max().item() * 2 ** 24


def test_float32_activations_keep_their_digits():
    """silu and sigmoid of exact inputs from -80 to 80.  The exponential is
    good to two half steps, its sum with one, the quotient and the products
    round once each, and the exponential's error counts in full: 8 half
    steps."""
    z = torch.linspace(-80, 80, 4001, device=DEV)
    s = 1 / (1 + torch.exp(-z.double()))
    one = torch.ones(z.numel(), 1, device=DEV)
    y, _ = mixer.conv1d_causal_fwd(z[None], one, act="silu")
    assert _steps(y[0], z.double() * s) <= 8
    y = mixer.conv1d_causal_step(z[None], one, None, torch.zeros(1, 0, z.numel(), device=DEV), act="silu")
    assert _steps(y[0], z.double() * s) <= 8
    # rows of one value: y / rms(y) is 1 (eps = 0), so r is act(gate), and dgate its slope
    yy, gate, w = torch.ones(z.numel(), 1, device=DEV), z[:, None].contiguous(), torch.ones(1, device=DEV)
    for act, want, slope in (("silu", z.double() * s, s * (1 + z.double() * (1 - s))), ("sigmoid", s, s * (1 - s))):
        r, _, stats = mixer.branch_norm_fwd(None, yy, w, gate, act=act, eps=0.0, save=True)
        assert _steps(r[:, 0], want) <= 8, act
        grads = mixer.branch_norm_bwd(yy, None, None, yy, w, gate, None, stats, act=act, eps=0.0)
        # below zero the slope is a product of what is accurate; above, 1 - s is a difference
        low = z < -2
        assert _steps(grads[3][low, 0], slope[low]) <= 24, act


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_at_the_ends_of_the_range(dtype):
    t, inf, nan = T16[dtype], float("inf"), float("nan")
    z = torch.tensor([inf, 3e38, 100.0, 0.0, -100.0, -3e38, nan], device=DEV).to(t)
    one = torch.ones(7, 1, device=DEV, dtype=t)
    y, _ = mixer.conv1d_causal_fwd(z[None], one, act="silu")
    assert (y[0, :3] == z[:3]).all() and y[0, 3] == 0 and (y[0, 4:6].float().abs() < 1e-37).all() and y[0, 6].isnan()
    z[5] = -inf
    r, _, _ = mixer.branch_norm_fwd(None, one, one[:1, 0], z[:, None].contiguous(), act="sigmoid", eps=0.0)
    assert (r[:3] == 1).all() and r[3] == 0.5 and (r[4:6].float() < 1e-37).all() and r[6].isnan()


# -------------------------------------------------------------- without rows


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_branch_norm_without_rows_but_with_a_gate(dtype):
    """The gated norm of no tokens: a gate row for each of no rows, or a gate
    that all would share."""
    t = T16[dtype]
    w = torch.ones(64, device=DEV, dtype=t)
    y = torch.zeros(0, 64, device=DEV, dtype=t)
    some = torch.zeros(4, 64, device=DEV, dtype=t)[:0]  # no rows of a buffer that is there
    for gate in (y, some):
        r, h, stats = mixer.branch_norm_fwd(y, y, w, gate, w, act="silu", save=True)
        assert r.shape == h.shape == (0, 64)
        grads = mixer.branch_norm_bwd(y, y, y, y, w, gate, w, stats, act="silu")
        assert grads[3].shape == (0, 64)
        assert (grads[2] == 0).all() and (grads[4] == 0).all()
    gate = torch.ones(1, 64, device=DEV, dtype=t)
    r, h, stats = mixer.branch_norm_fwd(y, y, w, gate, w, act="silu", save=True)
    grads = mixer.branch_norm_bwd(y, y, y, y, w, gate, w, stats, act="silu")
    assert all((z == 0).all() for z in grads[2:])
    leaves = [z.clone().requires_grad_(True) for z in (y, w, y)]
    r, _ = mixer.branch_norm(None, leaves[0], leaves[1], leaves[2], act="silu")
    assert [z.shape for z in torch.autograd.grad(r.sum(), leaves)] == [z.shape for z in leaves]
    with pytest.raises(ValueError):  # no gate rows for rows that are there
        mixer.branch_norm_fwd(None, torch.ones(2, 64, device=DEV, dtype=t), w, gate[:0])
