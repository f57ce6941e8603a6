"""Host-side checks of the sequence-mixing operators (no GPU: nothing here
launches a kernel), and the 64-bit definitions against finite differences."""
import ctypes
import os
import re

import pytest
import torch

import convolution_lowering_amd as cl
from convolution_lowering_amd import mixer
from oracle import mixer as om

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "convlower_mixer.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below is refused on the host
ODD = ctypes.c_void_p(0x1001)


def L():
    return mixer._mixer_lib()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^conv_status_t\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(mixer.EXPORTS)
    for n in names:
        assert hasattr(cl.lib(), n), n
    for macro, value in (("MIX_CONV1D_MAX_WIDTH", mixer.MAX_CONV_WIDTH), ("MIX_DELTA_MAX_DK", mixer.MAX_DK),
                         ("MIX_DELTA_MAX_DV", mixer.MAX_DV), ("MIX_NORM_MAX_WIDTH", mixer.MAX_NORM_WIDTH)):
        assert int(re.search(rf"#define {macro} (\d+)", text).group(1)) == value


def conv_fwd(x=P, xs=64, w=P, bias=None, state=None, cu=None, y=P, out=None, T=8, N=1, D=64, W=4, act=1, dt=1):
    return L().conv1d_causal_fwd(x, xs, w, bias, state, cu, y, out, T, N, D, W, act, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x=ODD), INVALID),
    (dict(state=ODD), INVALID), (dict(cu=ODD), INVALID), (dict(xs=63), INVALID), (dict(D=0), INVALID),
    (dict(W=0), INVALID), (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(T=7, N=2), INVALID),
    (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(dt=3), INVALID), (dict(dt=9), INVALID),
    (dict(W=9), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
])
def test_conv_fwd_refusals(bad, want):
    assert conv_fwd(**bad) == want


def conv_bwd(dy=P, dys=64, x=P, xs=64, w=P, bias=None, dx=P, dw=P, db=None, T=8, N=1, D=64, W=4, ws=P, nbytes=1 << 20):
    return L().conv1d_causal_bwd(dy, dys, None, x, xs, w, bias, None, None, dx, dw, db, None, T, N, D, W, 1, 1, None, ws,
                                 nbytes)


@pytest.mark.parametrize("bad,want", [
    (dict(dy=None), INVALID), (dict(dys=1), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(db=P), INVALID), (dict(ws=None), WORKSPACE), (dict(nbytes=4), WORKSPACE), (dict(ws=ODD), INVALID),
    (dict(W=9), UNSUPPORTED),
])
def test_conv_bwd_refusals(bad, want):
    assert conv_bwd(**bad) == want


def conv_step(x=P, xs=64, w=P, pool=P, slots=P, y=P, R=2, Pn=4, D=64, W=4, act=1, dt=1):
    return L().conv1d_causal_step(x, xs, w, None, pool, slots, y, R, Pn, D, W, act, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(pool=None), INVALID), (dict(slots=ODD), INVALID), (dict(R=-1), INVALID),
    (dict(slots=None, R=5), INVALID), (dict(xs=3), INVALID), (dict(R=0), OK), (dict(W=9), UNSUPPORTED),
])
def test_conv_step_refusals(bad, want):
    assert conv_step(**bad) == want


def delta_fwd(q=P, qs=256, k=P, ks=256, v=P, vs=512, g=P, beta=P, state=None, cu=None, o=P, T=8, N=1, Hk=2, Hv=4,
              dk=128, dv=128, dt=1, bdt=1, ws=P, nbytes=1 << 40, saved=None, saved_bytes=0):
    return L().delta_rule_fwd(q, qs, k, ks, v, vs, g, beta, state, cu, o, None, T, N, Hk, Hv, dk, dv, 1.0, 0, dt, bdt,
                              None, ws, nbytes, saved, saved_bytes)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(o=None), INVALID), (dict(q=ODD), INVALID), (dict(state=ODD), INVALID),
    (dict(qs=255), INVALID), (dict(vs=511), INVALID), (dict(Hv=3), INVALID), (dict(Hk=0), INVALID),
    (dict(dk=0), INVALID), (dict(dt=3), INVALID), (dict(bdt=2), INVALID), (dict(T=9, N=2), INVALID),
    (dict(dk=129, qs=400, ks=400), UNSUPPORTED), (dict(dv=257, vs=2000), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(vs=(1 << 22) + 1), UNSUPPORTED), (dict(Hv=40000, vs=40000 * 128), UNSUPPORTED), (dict(Hv=65536), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=8), WORKSPACE), (dict(saved=P, saved_bytes=8), WORKSPACE),
    (dict(ws=ODD), INVALID), (dict(saved=ODD, saved_bytes=1 << 40), INVALID),
])
def test_delta_fwd_refusals(bad, want):
    assert delta_fwd(**bad) == want


def delta_bwd(d_o=P, dos=512, q=P, qs=256, k=P, ks=256, v=P, vs=512, g=P, beta=P, cu=None, dst=None, dq=P, dk_=P, dv_=P,
              dg=P, dbeta=P, ds=None, T=8, N=1, Hk=2, Hv=4, dk=128, dv=128, dt=1, bdt=1, ws=P, nbytes=1 << 40, saved=P,
              saved_bytes=1 << 40):
    return L().delta_rule_bwd(d_o, dos, dst, q, qs, k, ks, v, vs, g, beta, cu, saved, saved_bytes, dq, dk_, dv_, dg,
                              dbeta, ds, T, N, Hk, Hv, dk, dv, 1.0, 0, dt, bdt, None, ws, nbytes)


@pytest.mark.parametrize("bad,want", [
    (dict(d_o=None), INVALID), (dict(d_o=ODD), INVALID), (dict(dos=511), INVALID), (dict(q=None), INVALID),
    (dict(dq=None), INVALID), (dict(dk_=None), INVALID), (dict(dv_=None), INVALID), (dict(dg=None), INVALID),
    (dict(dbeta=None), INVALID), (dict(dst=ODD), INVALID), (dict(ds=ODD), INVALID), (dict(ks=255), INVALID),
    (dict(ws=None), WORKSPACE), (dict(nbytes=8), WORKSPACE), (dict(saved=None), WORKSPACE), (dict(saved_bytes=8), WORKSPACE),
    (dict(dos=(1 << 22) + 1), UNSUPPORTED), (dict(dk=129, qs=400, ks=400), UNSUPPORTED),
])
def test_delta_bwd_refusals(bad, want):
    assert delta_bwd(**bad) == want


def delta_step(q=P, qs=256, v=P, vs=512, g=P, beta=P, pool=P, slots=P, o=P, R=2, Ln=1, Pn=4, Hk=2, Hv=4, dk=128, dv=128):
    return L().delta_rule_step(q, qs, q, qs, v, vs, g, beta, pool, slots, o, R, Ln, Pn, Hk, Hv, dk, dv, 1.0, 0, 1, 1, None)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), INVALID), (dict(pool=None), INVALID), (dict(pool=ODD), INVALID), (dict(slots=ODD), INVALID),
    (dict(R=-1), INVALID), (dict(Ln=-1), INVALID), (dict(slots=None, R=5), INVALID), (dict(qs=4), INVALID),
    (dict(Hv=5), INVALID), (dict(R=0), OK), (dict(Ln=0), OK), (dict(dk=130, qs=400), UNSUPPORTED),
    (dict(R=1 << 23, Hv=4), UNSUPPORTED),  # more wavefronts than a launch has
])
def test_delta_step_refusals(bad, want):
    assert delta_step(**bad) == want


def norm_fwd(x=P, y=P, wp=P, gate=None, wn=P, r=P, h=P, stats=None, R=4, D=64, G=4, eps=1e-6, act=0, dt=1):
    return L().branch_norm_fwd(x, y, wp, gate, wn, r, h, stats, R, D, G, 1.0, eps, act, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(y=None), INVALID), (dict(wp=None), INVALID), (dict(r=None), INVALID), (dict(h=None), INVALID),
    (dict(wn=None), INVALID), (dict(gate=P, G=3), INVALID), (dict(gate=P, G=0), INVALID), (dict(gate=P, G=8), INVALID),
    (dict(y=ODD), INVALID), (dict(stats=ODD), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(act=3), INVALID), (dict(dt=3), INVALID), (dict(D=0), INVALID), (dict(R=0), OK), (dict(D=32769), UNSUPPORTED),
])
def test_norm_fwd_refusals(bad, want):
    assert norm_fwd(**bad) == want


def norm_bwd(dr=P, dh=P, x=P, y=P, gate=None, wn=P, stats=P, dx=P, dy=P, dw=P, dgate=None, dwn=P, R=4, D=64, G=4, ws=P,
             nbytes=1 << 30):
    return L().branch_norm_bwd(dr, dh, x, y, P, gate, wn, stats, dx, dy, dw, dgate, dwn, R, D, G, 1.0, 1e-6, 0, 1, None,
                               ws, nbytes)


@pytest.mark.parametrize("bad,want", [
    (dict(dx=None), INVALID), (dict(x=None), INVALID), (dict(dgate=P), INVALID), (dict(gate=P), INVALID),
    (dict(dwn=None), INVALID), (dict(wn=None, dwn=None), INVALID), (dict(stats=None), INVALID), (dict(dw=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(nbytes=8), WORKSPACE),
])
def test_norm_bwd_refusals(bad, want):
    assert norm_bwd(**bad) == want


def test_size_queries():
    out = ctypes.c_size_t()
    assert L().conv1d_causal_bwd_workspace_size(1000, 3, 64, 4, None) == INVALID
    assert L().conv1d_causal_bwd_workspace_size(1000, 3, 64, 4, ctypes.byref(out)) == OK
    assert 0 < out.value < 1000 * 64 * 4
    assert L().conv1d_causal_bwd_workspace_size(0, 3, 64, 4, ctypes.byref(out)) == OK and out.value == 0
    for fn in (L().delta_rule_fwd_workspace_size, L().delta_rule_saved_size, L().delta_rule_bwd_workspace_size):
        assert fn(100, 2, 2, 4, 64, 64, 1, None) == INVALID
        assert fn(-1, 2, 2, 4, 64, 64, 1, ctypes.byref(out)) == INVALID
        assert fn(100, 2, 2, 3, 64, 64, 1, ctypes.byref(out)) == INVALID
        assert fn(100, 2, 2, 4, 300, 64, 1, ctypes.byref(out)) == UNSUPPORTED
        assert fn(100, 2, 2, 4, 64, 64, 1, ctypes.byref(out)) == OK
    assert L().branch_norm_bwd_workspace_size(64, 128, 1, ctypes.byref(out)) == OK and out.value > 0
    assert L().branch_norm_bwd_workspace_size(64, 128, 5, ctypes.byref(out)) == INVALID


def test_binding_checks_before_the_library():
    x, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(64, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        mixer.conv1d_causal_fwd(x, w)
    with pytest.raises(TypeError):
        mixer.conv1d_causal_fwd(x.to(torch.float64), w)
    with pytest.raises(ValueError):
        mixer.conv1d_causal_fwd(x[:, :32], w)
    with pytest.raises(ValueError):
        mixer._act("gelu")
    with pytest.raises(ValueError):  # 3 value heads over 2 key heads
        mixer._delta_args(torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.zeros(4, 3, 8), None, torch.zeros(4, 3))
    with pytest.raises(ValueError):
        mixer._packing((2, 8), torch.zeros(3, dtype=torch.int32), x.device)
    with pytest.raises(ValueError):
        mixer._packing((8,), torch.zeros(3, dtype=torch.int64), x.device)


def _differences(fn, leaves, h=1e-6):
    """Central differences of a scalar function at a few places of each leaf."""
    for t in leaves:
        flat = t.detach().view(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 5)):
            old = flat[i].item()
            flat[i] = old + h
            up = fn().item()
            flat[i] = old - h
            down = fn().item()
            flat[i] = old
            yield t, i, (up - down) / (2 * h)


@pytest.mark.parametrize("op", ["conv", "delta", "norm"])
def test_definitions_differentiate(op):
    """autograd through the definitions against central differences: a step
    of 1e-6 leaves about 1e-10 of rounding and 1e-12 of curvature."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True)
    if op == "conv":
        leaves = [r(9, 3), r(3, 4), r(3), r(3, 3, 3)]
        fn = lambda: sum((o * o).sum() for o in om.conv1d_causal(*leaves[:3], [0, 2, 2, 9], leaves[3], "silu"))
    elif op == "delta":
        leaves = [r(6, 1, 4), r(6, 1, 4), r(6, 2, 3), r(6, 2), r(6, 2), r(2, 2, 4, 3)]
        fn = lambda: sum((o * o).sum() for o in om.delta_rule(leaves[0], leaves[1], leaves[2], -leaves[3].abs(), leaves[4],
                                                              [0, 1, 6], leaves[5], 0.7, True))
    else:
        leaves = [r(6, 5), r(6, 5), r(5), r(3, 5), r(5)]
        fn = lambda: sum((o * o).sum() for o in om.branch_norm(*leaves, 0.5, 1e-6, "silu"))
    grads = dict(zip(map(id, leaves), torch.autograd.grad(fn(), leaves)))
    with torch.no_grad():
        for t, i, d in _differences(fn, leaves):
            assert abs(grads[id(t)].view(-1)[i].item() - d) <= 1e-6 * (1 + abs(d))
