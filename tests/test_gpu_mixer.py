"""The sequence-mixing operators on the GPU against their 64-bit definitions.

Tolerances: a result rounded to type t is off by at most half a step,
finfo(t).eps / 2 of its value; before that n float32 roundings in series, of
at most 2^-24 of the largest result each.  n is counted for each operator
where it is passed.  For the delta rule, whose chunks multiply operands split
into two 11-bit halves (2^-22 of a product is lost) in at most 8 products in
series, 1e-5 of the result's norm stands for them.
"""
import pytest
import torch

from convolution_lowering_amd import mixer
from oracle import mixer as om

pytestmark = pytest.mark.gpu

DEV = "cuda"
T16 = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def _say(*a):
    print("[gpu]", *a, flush=True)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _close(got, ref, n, what):
    assert got.shape == ref.shape, what
    if not got.numel():
        return
    d, ref = got.double(), ref.double()
    assert torch.isfinite(d).all(), what
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    off = (d - ref).abs() - half * ref.abs()
    assert off.max() <= n * U * ref.abs().max() + tiny, f"{what}: {off.max():.3e} over, largest {ref.abs().max():.3e}"


def _near(got, ref, what, loose=1e-5):
    """2-norm: half a step of rounding, and `loose`."""
    assert got.shape == ref.shape, what
    if not got.numel():
        return
    d, ref = got.double(), ref.double()
    assert torch.isfinite(d).all(), what
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    assert (d - ref).norm() <= (half + loose) * ref.norm() + 1e-30, f"{what}: {(d - ref).norm() / ref.norm():.3e}"


# ------------------------------------------------------------ causal convolution

CONV = [  # lens (None: one sequence), D, W, dtype, bias, state, act, token padding
    ([5, 1, 0, 70, 3], 64, 4, "bf16", True, True, "silu", 0),
    ([5, 1, 0, 70, 3], 64, 4, "fp32", True, False, "silu", 64),
    ([1], 8, 4, "bf16", True, True, "silu", 0),
    ([300, 2, 200], 37, 4, "fp16", False, True, "none", 5),
    ([129], 2056, 3, "bf16", True, True, "silu", 8),
    ([64, 64, 64], 100, 2, "fp32", True, True, "silu", 0),
    ([33, 0, 7], 40, 1, "bf16", True, False, "silu", 0),
    ([3, 30, 1, 9], 72, 8, "fp16", True, True, "silu", 0),
    ([3, 30, 1, 9], 11, 6, "fp32", False, True, "none", 1),
    ([0, 0], 16, 4, "bf16", True, True, "silu", 0),
    ([700, 41], 264, 4, "bf16", True, True, "silu", 0),
]


def _conv_case(case, seed=5):
    lens, D, W, dtype, bias, state, act, pad = case
    g, t = _gen(seed), T16[dtype]
    T = sum(lens)
    wide = _randn(g, T, D + pad).to(t)
    x = wide[:, :D]
    return (x, _randn(g, D, W).to(t), _randn(g, D).to(t) if bias else None, _cu(lens),
            _randn(g, len(lens), W - 1, D).to(t) if state else None, act, g, t)


@pytest.mark.parametrize("case", CONV, ids=[f"{c[3]}-D{c[1]}-W{c[2]}-{len(c[0])}seq" for c in CONV])
def test_conv1d_forward_and_gradients(case):
    x, w, b, cu, state, act, g, t = _conv_case(case)
    T, D = x.shape
    W = w.shape[1]
    _say("conv1d", case)
    y, out = mixer.conv1d_causal_fwd(x, w, b, cu_seqlens=cu, state=state, act=act, want_state=True)
    leaves = [None if z is None else z.double().requires_grad_(True) for z in (x, w, b, state)]
    ry, rout = om.conv1d_causal(leaves[0], leaves[1], leaves[2], cu.tolist(), leaves[3], act)
    # W + 1 roundings of the sum; the exponential, the sigmoid and its product: under 32
    _close(y, ry.detach(), 32 + W, "y")
    assert torch.equal(out.double(), rout.detach())
    dy, dso = _randn(g, T, D).to(t), _randn(g, *out.shape).to(t)
    grads = mixer.conv1d_causal_bwd(dy, x, w, b, cu_seqlens=cu, state=state, act=act, dstate_out=dso,
                                    want_dstate=True)
    total = (ry * dy.double()).sum() + (rout * dso.double()).sum()
    need = [z for z in leaves if z is not None]
    ref = dict(zip(map(id, need), torch.autograd.grad(total, need, allow_unused=True)))
    ref = [None if z is None else ref[id(z)] if ref[id(z)] is not None else torch.zeros_like(z) for z in leaves]
    _close(grads[0], ref[0], 64 + 2 * W, "dx")
    # sums over T tokens
    _close(grads[1], ref[1], 64 + T, "dw")
    if b is None:
        assert grads[2] is None
    else:
        _close(grads[2], ref[2], 64 + T, "dbias")
    if state is not None:
        _close(grads[3], ref[3], 64 + 2 * W, "dstate")
    else:
        assert torch.isfinite(grads[3].double()).all()


def test_conv1d_batched_and_split_sequences_agree():
    """[B, L, D] is the packed call; a sequence cut in two with the state
    handed on gives the bits of the whole."""
    g = _gen(1)
    x, w, b = _randn(g, 3, 50, 24).bfloat16(), _randn(g, 24, 4).bfloat16(), _randn(g, 24).bfloat16()
    y, s = mixer.conv1d_causal_fwd(x, w, b, want_state=True)
    yp, sp = mixer.conv1d_causal_fwd(x.reshape(150, 24), w, b, cu_seqlens=_cu([50, 50, 50]), want_state=True)
    assert torch.equal(y.reshape(150, 24), yp) and torch.equal(s, sp)
    y1, s1 = mixer.conv1d_causal_fwd(x[:, :17].contiguous(), w, b, want_state=True)
    y2, s2 = mixer.conv1d_causal_fwd(x[:, 17:].contiguous(), w, b, state=s1, want_state=True)
    assert torch.equal(torch.cat((y1, y2), 1), y) and torch.equal(s2, s)


@pytest.mark.parametrize("D,W,dtype", [(64, 4, "bf16"), (2056, 4, "fp16"), (37, 3, "fp32"), (8, 1, "bf16"), (100, 8, "bf16")])
def test_conv1d_step_continues_the_sequence(D, W, dtype):
    g, t = _gen(2), T16[dtype]
    x, w, b = _randn(g, 4, 12, D).to(t), _randn(g, D, W).to(t), _randn(g, D).to(t)
    ref, _ = om.conv1d_causal(x.double().reshape(48, D), w.double(), b.double(), [0, 12, 24, 36, 48], None, "silu")
    pool = torch.full((7, W - 1, D), 9.0, device=DEV, dtype=t)
    slots = torch.tensor([5, 0, 2, 3], dtype=torch.int32, device=DEV)
    pool[slots.long()] = 0
    for i in range(12):
        y = mixer.conv1d_causal_step(x[:, i], w, b, pool, slots)
        _close(y, ref.reshape(4, 12, D)[:, i], 32 + W, f"token {i}")
    if W > 1:
        keep = torch.cat((torch.zeros_like(x[:, :8]), x), 1)[:, -(W - 1):]
        assert torch.equal(pool[slots.long()], keep)
        assert (pool[[1, 4, 6]] == 9).all()
    bad = torch.tensor([-1, 7, 2, 1 << 30], dtype=torch.int32, device=DEV)
    before = pool.clone()
    y = mixer.conv1d_causal_step(x[:, 0], w, b, pool, bad)
    assert (y[[0, 1, 3]] == 0).all()
    changed = [2]
    rest = [i for i in range(7) if i not in changed]
    assert torch.equal(pool[rest], before[rest])


# -------------------------------------------------------------- gated delta rule


def _delta_inputs(lens, Hk, Hv, dk, dv, dtype, seed=7, packed=True, beta32=False, fast=1.0):
    g, t = _gen(seed), T16[dtype]
    T = sum(lens)
    mixed = torch.nn.functional.silu(_randn(g, T, 2 * Hk * dk + Hv * dv)).to(t)
    q, k, v = mixed.split((Hk * dk, Hk * dk, Hv * dv), -1)
    q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    gate = -fast * torch.exp(_randn(g, T, Hv) * 2 - 3)
    beta = torch.sigmoid(_randn(g, T, Hv)).to(torch.float32 if beta32 else t)
    return q, k, v, gate, beta, g


def _delta_ref(q, k, v, gate, beta, cu, state, scale, qk_norm):
    return om.delta_rule(q.double(), k.double(), v.double(), gate.double(), beta.double(), cu,
                         None if state is None else state.double(), scale, qk_norm)


DELTA = [  # lens, Hk, Hv, dk, dv, dtype, state, packed, fp32 beta
    ([1], 1, 1, 128, 128, "bf16", True, False, False),
    ([1, 0, 64, 65, 63], 1, 2, 128, 128, "bf16", True, True, False),
    ([200, 17], 2, 2, 64, 64, "fp32", True, True, False),
    ([130], 2, 6, 72, 100, "fp32", False, True, False),
    ([129, 5], 3, 3, 40, 33, "fp16", True, True, True),
    ([77], 1, 1, 1, 1, "bf16", True, False, True),
    ([300], 1, 4, 128, 256, "bf16", False, True, False),
    ([40, 90], 1, 2, 100, 130, "fp16", True, False, False),
    ([700, 64, 321], 2, 2, 128, 80, "bf16", True, True, False),
    ([400], 1, 3, 128, 128, "fp32", True, True, False),
]


@pytest.mark.parametrize("case", DELTA, ids=[f"{c[5]}-{c[1]}x{c[2]}-{c[3]}x{c[4]}-{sum(c[0])}tok" for c in DELTA])
def test_delta_rule_forward(case):
    lens, Hk, Hv, dk, dv, dtype, has_state, packed, b32 = case
    _say("delta fwd", case)
    q, k, v, gate, beta, g = _delta_inputs(lens, Hk, Hv, dk, dv, dtype, packed=packed, beta32=b32)
    cu = _cu(lens)
    state = _randn(g, len(lens), Hv, dk, dv) * 0.3 if has_state else None
    o, s, _ = mixer.delta_rule_fwd(q, k, v, gate, beta, cu_seqlens=cu, state=state, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(q, k, v, gate, beta, cu.tolist(), state, dk ** -0.5, True)
    _near(o, ro, "o")
    _near(s, rs, "state")


@pytest.mark.parametrize("L,rows,dk,dv,dtype", [(1, 5, 128, 128, "bf16"), (6, 2, 128, 96, "bf16"), (3, 2, 64, 64, "fp16"), (2, 3, 100, 30, "fp32"),
                                                 (1, 1, 17, 7, "bf16")])
def test_delta_rule_step_continues_the_sequence(L, rows, dk, dv, dtype):
    Hk, Hv, steps = 2, 4, 4
    q, k, v, gate, beta, g = _delta_inputs([rows * L * steps], Hk, Hv, dk, dv, dtype)
    view = lambda z: z.unflatten(0, (rows, steps * L))
    q, k, v, gate, beta = map(view, (q, k, v, gate, beta))
    pool = _randn(g, rows + 3, Hv, dk, dv)
    slots = torch.randperm(rows + 3, generator=g, device=DEV)[:rows].to(torch.int32)
    before = pool.clone()
    refs = [_delta_ref(q[r], k[r], v[r], gate[r], beta[r], None, before[slots[r]][None], 0.25, True) for r in range(rows)]
    outs = []
    for i in range(steps):
        at = slice(i * L, (i + 1) * L)
        args = [z[:, at].contiguous() for z in (q, k, v, gate, beta)]
        if L == 1:
            args = [z.squeeze(1) for z in args]
        outs.append(mixer.delta_rule_step(*args, pool, slots, scale=0.25, qk_norm=True).reshape(rows, L, Hv, dv))
    _near(torch.cat(outs, 1), torch.stack([r[0] for r in refs]), "o")
    _near(pool[slots.long()], torch.cat([r[1] for r in refs]), "pool")
    rest = [i for i in range(rows + 3) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_delta_rule_step_padding_requests():
    q, k, v, gate, beta, g = _delta_inputs([3], 1, 2, 64, 64, "bf16")
    pool = _randn(g, 2, 2, 64, 64)
    before = pool.clone()
    o = mixer.delta_rule_step(q, k, v, gate, beta, pool, torch.tensor([-1, 1, 2], dtype=torch.int32, device=DEV))
    assert (o[[0, 2]] == 0).all() and (o[1] != 0).any()
    assert torch.equal(pool[0], before[0]) and not torch.equal(pool[1], before[1])


def _delta_grads(case, seed=7, fast=1.0):
    lens, Hk, Hv, dk, dv, dtype, has_state, packed, b32 = case
    q, k, v, gate, beta, g = _delta_inputs(lens, Hk, Hv, dk, dv, dtype, packed=packed, beta32=b32, seed=seed, fast=fast)
    cu = _cu(lens)
    state = _randn(g, len(lens), Hv, dk, dv) * 0.3 if has_state else None
    do = _randn(g, sum(lens), Hv, dv).to(q.dtype)
    ds = _randn(g, len(lens), Hv, dk, dv) * 0.3 if has_state else None
    return q, k, v, gate, beta, cu, state, do, ds


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "raw"])
@pytest.mark.parametrize("case", DELTA, ids=[f"{c[5]}-{c[1]}x{c[2]}-{c[3]}x{c[4]}-{sum(c[0])}tok" for c in DELTA])
def test_delta_rule_gradients(case, norm):
    _say("delta bwd", case, norm)
    q, k, v, gate, beta, cu, state, do, ds = _delta_grads(case)
    if not norm:  # keys no longer than one, as the rule needs
        k = (k.float() * 0.7 / k.float().norm(dim=-1).amax().clamp(min=1e-3)).to(k.dtype)
    more = dict(cu_seqlens=cu, scale=0.3, qk_norm=norm)
    o, s, saved = mixer.delta_rule_fwd(q, k, v, gate, beta, state=state, want_state=True, save=True, **more)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, gate, beta)]
    rstate = None if state is None else state.double().requires_grad_(True)
    ro, rs = om.delta_rule(*leaves, cu.tolist(), rstate, 0.3, norm)
    _near(o, ro.detach(), "o")
    _near(s, rs.detach(), "state")
    total = (ro * do.double()).sum()
    if ds is not None:
        total = total + (rs * ds.double()).sum()
    ref = torch.autograd.grad(total, leaves + ([rstate] if rstate is not None else []))
    got = mixer.delta_rule_bwd(do, q, k, v, gate, beta, saved, dstate_out=ds, want_dstate=state is not None, **more)
    # one key of one value: with the norm, q and k are +-1 and their gradients the eps of the norm away from nothing
    names = ("dq", "dk", "dv", "dg", "dbeta", "dstate")
    for name, x, y in zip(names, got, ref):
        if case[3] == 1 and norm and name in ("dq", "dk"):
            assert torch.isfinite(x.float()).all()
            continue
        _near(x, y, name, 2e-5)  # forward and backward in series
    if state is None:
        assert got[5] is None


def test_delta_rule_strong_and_cleared_decays():
    """Decays from none to a cleared state (-inf) side by side."""
    case = ([150, 64, 3], 2, 4, 128, 64, "fp32", True, True, True)
    q, k, v, gate, beta, cu, state, do, ds = _delta_grads(case)
    r = torch.rand(gate.shape, generator=_gen(3), device=DEV)
    gate = torch.where(r < 0.1, -60.0, torch.where(r < 0.2, 0.0, torch.where(r < 0.25, -300.0, gate)))
    soft = gate.clone()
    gate = torch.where((r > 0.5) & (r < 0.53), -float("inf"), gate)
    hard = torch.where((r > 0.5) & (r < 0.53), -5000.0, soft)  # e^-5000 is zero in 64 bits as well
    more = dict(cu_seqlens=cu, scale=1.0, qk_norm=True)
    o, s, saved = mixer.delta_rule_fwd(q, k, v, gate, beta, state=state, want_state=True, save=True, **more)
    leaves = [z.double().requires_grad_(True) for z in (q, k, v, hard, beta, state)]
    ro, rs = om.delta_rule(*leaves[:5], cu.tolist(), leaves[5], 1.0, True)
    _near(o, ro.detach(), "o")
    _near(s, rs.detach(), "state")
    ref = torch.autograd.grad((ro * do.double()).sum() + (rs * ds.double()).sum(), leaves)
    got = mixer.delta_rule_bwd(do, q, k, v, gate, beta, saved, dstate_out=ds, want_dstate=True, **more)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), got, ref):
        _near(x, y, name, 2e-5)


def test_delta_rule_repeated_keys():
    """Every key of a chunk the same: the chunk's matrix is as far from 1 as
    it gets, with beta = 1 and no decay."""
    g = _gen(4)
    k = _randn(g, 1, 1, 128).expand(100, 1, 128).contiguous()
    q, v = _randn(g, 100, 1, 128), _randn(g, 100, 1, 128)
    gate, beta = torch.zeros(100, 1, device=DEV), torch.ones(100, 1, device=DEV)
    o, s, _ = mixer.delta_rule_fwd(q, k, v, gate, beta, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(q, k, v, gate, beta, None, None, 128 ** -0.5, True)
    _near(o, ro, "o")
    _near(s, rs, "state")


@pytest.mark.parametrize("mag", [1e-6, 1.0, 3e4])
def test_delta_rule_magnitudes(mag):
    """Values, states and keys far from one: the powers of two that move
    operands into f16's range."""
    g = _gen(6)
    q, k, v = (_randn(g, 90, 2, 64).bfloat16() for _ in range(3))
    v, k = v * mag, k * mag
    gate, beta = -torch.rand(90, 2, generator=g, device=DEV), torch.sigmoid(_randn(g, 90, 2)).bfloat16()
    state = _randn(g, 1, 2, 64, 64) * mag
    o, s, _ = mixer.delta_rule_fwd(q, k, v, gate, beta, state=state, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(q, k, v, gate, beta, None, state, 0.125, True)
    _near(o, ro, "o")
    _near(s, rs, "state")


def test_delta_rule_sequences_cut_and_batched():
    """[B, L] is the packed call; a sequence cut anywhere, its state handed
    on, continues (in the token form too)."""
    q, k, v, gate, beta, g = _delta_inputs([300], 2, 4, 128, 128, "bf16")
    args = (q, k, v, gate, beta)
    o, s, _ = mixer.delta_rule_fwd(*args, qk_norm=True, want_state=True)
    ro, rs = _delta_ref(*args, None, None, 128 ** -0.5, True)
    head = [z[:131].contiguous() for z in args]
    o1, s1, _ = mixer.delta_rule_fwd(*head, qk_norm=True, want_state=True)
    o2, s2, _ = mixer.delta_rule_fwd(*[z[131:] for z in args[:3]], gate[131:], beta[131:], state=s1, qk_norm=True,
                                     want_state=True)
    _near(torch.cat((o1, o2)), ro, "cut")
    _near(s2, rs, "cut state")
    pool = s1.clone()
    one = [z[131:134].contiguous()[None] for z in args]
    ot = mixer.delta_rule_step(*one, pool, qk_norm=True)
    _near(ot[0], ro[131:134], "continued by tokens")
    batched = [z.unflatten(0, (3, 100)) for z in args]
    ob, sb, _ = mixer.delta_rule_fwd(*batched, qk_norm=True, want_state=True)
    op, sp, _ = mixer.delta_rule_fwd(*args, cu_seqlens=_cu([100, 100, 100]), qk_norm=True, want_state=True)
    assert torch.equal(ob.flatten(0, 1), op) and torch.equal(sb, sp)


def test_delta_rule_without_tokens():
    q = torch.zeros(0, 1, 64, device=DEV, dtype=torch.bfloat16)
    g = torch.zeros(0, 1, device=DEV)
    state = torch.randn(2, 1, 64, 64, device=DEV)
    o, s, saved = mixer.delta_rule_fwd(q, q, q, g, g, cu_seqlens=_cu([0, 0]), state=state, want_state=True, save=True)
    assert o.shape == (0, 1, 64) and torch.equal(s, state)
    got = mixer.delta_rule_bwd(q, q, q, q, g, g, saved, cu_seqlens=_cu([0, 0]), dstate_out=state, want_dstate=True)
    assert torch.equal(got[5], state)


def test_delta_rule_twice_the_same_bits():
    case = ([200, 31], 2, 4, 128, 128, "bf16", True, True, False)
    q, k, v, gate, beta, cu, state, do, ds = _delta_grads(case)
    runs = []
    for _ in range(2):
        o, s, saved = mixer.delta_rule_fwd(q, k, v, gate, beta, cu_seqlens=cu, state=state, qk_norm=True,
                                           want_state=True, save=True)
        runs.append((o, s, *mixer.delta_rule_bwd(do, q, k, v, gate, beta, saved, cu_seqlens=cu, qk_norm=True,
                                                 dstate_out=ds, want_dstate=True)))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ------------------------------------------------------------------ all together


def _block(x, p, fn):
    """conv -> delta rule -> gated head norm -> residual and next norm."""
    T = x.shape[0]
    m, _ = fn.conv1d_causal(x, p["w"], p["b"], cu_seqlens=p["cu"])
    q, k, v = m.split((128, 128, 256), -1)
    o, _ = fn.delta_rule(q.unflatten(1, (2, 64)), k.unflatten(1, (2, 64)), v.unflatten(1, (4, 64)), p["g"], p["beta"],
                         cu_seqlens=p["cu"], qk_norm=True)
    u, _ = fn.branch_norm(None, o.reshape(T * 4, 64), p["wn"], p["z"], act="silu")
    return fn.branch_norm(p["x0"], u.reshape(T, 256), p["wp"], p["gate"], p["w2"], alpha=0.5)


def _block_params(T, t, g):
    r = lambda *s: _randn(g, *s).to(t)
    return dict(w=r(512, 4), b=r(512), cu=_cu([T - 40, 40]), g=-torch.rand(T, 4, generator=g, device=DEV),
                beta=torch.sigmoid(_randn(g, T, 4)).to(t), wn=r(64), z=r(T * 4, 64), x0=r(T, 256), wp=r(256),
                gate=r(1, 256), w2=r(256))


def test_autograd_through_the_operators_together():
    """Gradients of a whole mixer by autograd against those of the 64-bit
    definitions: float32, whose five steps in series stay within 1e-4."""
    g = _gen(9)
    p = _block_params(150, torch.float32, g)
    x = _randn(g, 150, 512)
    names = ["w", "b", "g", "beta", "wn", "z", "x0", "wp", "gate", "w2"]
    leaves = [x.requires_grad_(True)] + [p[n].requires_grad_(True) for n in names]
    r, h = _block(x, p, mixer)
    dr, dh = _randn(g, 150, 256), _randn(g, 150, 256)
    got = torch.autograd.grad((r, h), leaves, (dr, dh))

    class Ref:
        conv1d_causal = staticmethod(lambda x, w, b, cu_seqlens: om.conv1d_causal(x, w, b, cu_seqlens, None, "silu"))
        delta_rule = staticmethod(lambda q, k, v, g, b, cu_seqlens, qk_norm:
                                  om.delta_rule(q, k, v, g, b, cu_seqlens, None, 64 ** -0.5, True))
        branch_norm = staticmethod(lambda x, y, wp, gate, wn=None, alpha=1.0, act="none":
                                   om.branch_norm(x, y, wp, gate, wn, alpha, 1e-6, act))

    pd = {n: z.detach().double().requires_grad_(n in names) if z.is_floating_point() else z.tolist() for n, z in p.items()}
    xd = x.detach().double().requires_grad_(True)
    rr, rh = _block(xd, pd, Ref)
    ref = torch.autograd.grad((rr, rh), [xd] + [pd[n] for n in names], (dr.double(), dh.double()))
    _near(r.detach(), rr.detach(), "r", 1e-4)
    _near(h.detach(), rh.detach(), "h", 1e-4)
    for n, a, b in zip(["x"] + names, got, ref):
        _near(a, b, n, 1e-4)


def test_operators_on_another_stream_and_in_a_graph():
    """The same bits on a side stream, and from a captured graph replayed with
    other inputs between eager work."""
    g = _gen(10)
    p = _block_params(200, torch.bfloat16, g)
    x = _randn(g, 200, 512).bfloat16()
    xs = [_randn(g, 200, 512).bfloat16() for _ in range(3)]
    with torch.no_grad():
        ref = [tuple(z.clone() for z in _block(y, p, mixer)) for y in xs]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            r, h = _block(xs[0], p, mixer)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(r, ref[0][0]) and torch.equal(h, ref[0][1])
        y, _ = mixer.conv1d_causal_fwd(x, p["w"], p["b"], cu_seqlens=p["cu"], stream=side)
        side.synchronize()
        assert torch.equal(y, mixer.conv1d_causal_fwd(x, p["w"], p["b"], cu_seqlens=p["cu"])[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r, h = _block(x, p, mixer)
        for i, y in enumerate(xs):
            x.copy_(y)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(r, ref[i][0]) and torch.equal(h, ref[i][1])
            _block(xs[0], p, mixer)


# ------------------------------------------------------------------- branch norm

NORM = [  # rows, D, gate rows, act, x, w_next, dtype
    (5, 4096, 5, "none", True, True, "bf16"),
    (1, 4000, 1, "sigmoid", True, True, "fp16"),
    (37, 128, 37, "silu", False, False, "bf16"),
    (37, 128, 1, "silu", True, True, "fp32"),
    (48, 200, 4, "none", True, True, "bf16"),
    (6, 8192, 0, "none", True, True, "bf16"),
    (3, 77, 3, "sigmoid", True, False, "fp16"),
    (9, 1, 1, "silu", False, True, "fp32"),
    (4, 5001, 2, "silu", True, True, "bf16"),
    (2, 32768, 1, "none", True, True, "bf16"),
    (600, 1032, 600, "silu", True, True, "bf16"),
    (2000, 256, 1, "none", True, True, "bf16"),
    (3, 9000, 1, "none", False, True, "fp32"),
]


@pytest.mark.parametrize("case", NORM, ids=[f"{c[6]}-{c[0]}x{c[1]}-gate{c[2]}-{c[3]}" for c in NORM])
def test_branch_norm_forward_and_gradients(case):
    R, D, G, act, has_x, has_next, dtype = case
    _say("branch norm", case)
    g, t = _gen(11), T16[dtype]
    y, w = _randn(g, R, D).to(t), (1 + 0.3 * _randn(g, D)).to(t)
    x = _randn(g, R, D).to(t) if has_x else None
    gate = _randn(g, G, D).to(t) if G else None
    wn = (1 + 0.3 * _randn(g, D)).to(t) if has_next else None
    r, h, stats = mixer.branch_norm_fwd(x, y, w, gate, wn, alpha=0.5, act=act, save=True)
    leaves = [None if z is None else z.double().requires_grad_(True) for z in (x, y, w, gate, wn)]
    rr, rh = om.branch_norm(*leaves, 0.5, 1e-6, act)
    # a row's sum: at most 32 additions in a thread and 10 between threads; twice, and 40 for the rest
    _close(r, rr.detach(), 128, "r")
    dr, dh = _randn(g, R, D).to(t), _randn(g, R, D).to(t) if has_next else None
    total = (rr * dr.double()).sum()
    if has_next:
        _close(h, rh.detach(), 128, "h")
        total = total + (rh * dh.double()).sum()
    else:
        assert h is None
    grads = mixer.branch_norm_bwd(dr, dh, x, y, w, gate, wn, stats, alpha=0.5, act=act)
    need = [z for z in leaves if z is not None]
    ref = dict(zip(map(id, need), torch.autograd.grad(total, need)))
    for name, got, leaf in zip(("dx", "dy", "dw_post", "dgate", "dw_next"), grads, leaves):
        if leaf is None:
            assert got is None
            continue
        rows = R if name.startswith("dw") else R // G if name == "dgate" else 0
        # D = 1: dy is the difference of equal numbers, eps apart; what is left is judged against what cancels
        if D == 1 and name in ("dy", "dx"):
            assert (got.double() - ref[id(leaf)]).abs().max() <= 128 * U * dr.abs().max() * 8
            continue
        _close(got, ref[id(leaf)], 256 + rows, name)


@pytest.mark.parametrize("R,D,dtype", [(9, 1024, "bf16"), (70, 41, "fp16"), (3, 4099, "fp32"), (5, 7, "bf16")])
def test_branch_norm_at_any_address(R, D, dtype):
    """Rows that begin one, two or three values past a 16-byte boundary."""
    _say("branch norm, any address", R, D, dtype)
    g, t = _gen(13), T16[dtype]

    def at(off, *shape):
        n = torch.Size(shape).numel()
        return torch.full((n + 16,), 7.0, device=DEV).to(t)[off:off + n].view(shape).copy_(_randn(g, *shape).to(t))

    y, x, gate, w, wn = at(1, R, D), at(2, R, D), at(3, R, D), at(1, D), at(0, D)
    dr, dh = at(3, R, D), at(1, R, D)
    leaves = [z.double().requires_grad_(True) for z in (x, y, w, gate, wn)]
    rr, rh = om.branch_norm(*leaves, 0.5, 1e-6, "silu")
    r, h, stats = mixer.branch_norm_fwd(x, y, w, gate, wn, alpha=0.5, act="silu", save=True)
    _close(r, rr.detach(), 128, "r")
    _close(h, rh.detach(), 128, "h")
    ref = torch.autograd.grad((rr * dr.double()).sum() + (rh * dh.double()).sum(), leaves)
    grads = mixer.branch_norm_bwd(dr, dh, x, y, w, gate, wn, stats, alpha=0.5, act="silu")
    for name, got, z in zip(("dx", "dy", "dw_post", "dgate", "dw_next"), grads, ref):
        _close(got, z, 256 + (R if name.startswith("dw") else 0), name)


def test_branch_norm_without_rows_and_without_gradients():
    w = torch.ones(64, device=DEV, dtype=torch.bfloat16)
    y = torch.zeros(0, 64, device=DEV, dtype=torch.bfloat16)
    r, h, stats = mixer.branch_norm_fwd(y, y, w, None, w, save=True)
    assert r.shape == h.shape == (0, 64)
    grads = mixer.branch_norm_bwd(y, y, y, y, w, None, w, stats)
    assert (grads[2] == 0).all() and (grads[4] == 0).all()
    y = torch.randn(5, 64, device=DEV).bfloat16()
    r, h, stats = mixer.branch_norm_fwd(y, y, w, None, w, save=True)
    grads = mixer.branch_norm_bwd(None, None, y, y, w, None, w, stats)
    assert all((z == 0).all() for z in grads if z is not None)
