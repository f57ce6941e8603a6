"""Host-side checks of the feed-forward operators (no GPU: nothing here launches
a kernel), and the 64-bit definitions against finite differences."""
import ctypes
import os
import re

import pytest
import torch

import convolution_lowering_amd as cl
from convolution_lowering_amd import ffn
from oracle import ffn as of
from test_mixer_boundary import _differences

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "convlower_ffn.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below is refused on the host, or has nothing to do
ODD = ctypes.c_void_p(0x1001)
BIG = 1 << 45


def L():
    return ffn._ffn_lib()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^conv_status_t\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(ffn.EXPORTS)
    for n in names:
        assert hasattr(cl.lib(), n), n
    assert "#define FFN_MAX_WIDTH (1 << 20)" in text and ffn.MAX_WIDTH == 1 << 20
    assert int(re.search(r"#define FFN_MAX_NORM_WIDTH (\d+)", text).group(1)) == ffn.MAX_NORM_WIDTH
    codes = dict(re.findall(r"FFN_ACT_(\w+) = (\d)", text))
    assert {k.lower(): int(v) for k, v in codes.items()} == ffn.ACTS


def fwd(x=P, xs=64, wg=P, wu=P, h=P, saved=None, sb=0, T=8, D=64, F=32, act=1, dt=1):
    return L().gated_ffn_fwd(x, xs, wg, wu, h, saved, sb, T, D, F, act, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(wg=None), INVALID), (dict(wu=None), INVALID), (dict(h=None), INVALID),
    (dict(x=ODD), INVALID), (dict(wg=ODD), INVALID), (dict(wu=ODD), INVALID), (dict(h=ODD), INVALID),
    (dict(saved=ctypes.c_void_p(0x1004), sb=BIG), INVALID), (dict(saved=P, sb=8 * 2 * 32 * 4 - 1), WORKSPACE),
    (dict(xs=63), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID), (dict(T=-1), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(dt=3), INVALID), (dict(dt=-1), INVALID),
    (dict(D=(1 << 20) + 1, xs=1 << 21), UNSUPPORTED), (dict(xs=(1 << 20) + 1), UNSUPPORTED),
    (dict(F=(1 << 20) + 1), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=0), OK), (dict(T=0, x=None, h=None), OK),
    (dict(T=(1 << 31) - 300, F=1 << 20), UNSUPPORTED),  # more blocks than a launch has
])
def test_fwd_refusals(bad, want):
    assert fwd(**bad) == want


def bwd(dh=P, dhs=32, x=P, xs=64, wg=P, wu=P, saved=P, sb=BIG, dx=P, dwg=P, dwu=P, T=8, D=64, F=32, act=1, dt=1, ws=P,
        nbytes=BIG):
    return L().gated_ffn_bwd(dh, dhs, x, xs, wg, wu, saved, sb, dx, dwg, dwu, T, D, F, act, dt, None, ws, nbytes)


@pytest.mark.parametrize("bad,want", [
    (dict(dh=None), INVALID), (dict(x=None), INVALID), (dict(wg=None), INVALID), (dict(wu=None), INVALID),
    (dict(dx=None), INVALID), (dict(dwg=None), INVALID), (dict(dwu=None), INVALID), (dict(dh=ODD), INVALID),
    (dict(dx=ODD), INVALID), (dict(dhs=31), INVALID), (dict(xs=63), INVALID), (dict(dhs=(1 << 20) + 1), UNSUPPORTED),
    (dict(act=9), INVALID), (dict(dt=3), INVALID), (dict(saved=None), WORKSPACE), (dict(sb=64), WORKSPACE),
    (dict(saved=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(nbytes=64), WORKSPACE), (dict(ws=ODD), INVALID),
    (dict(T=-1), INVALID), (dict(F=0), INVALID), (dict(D=(1 << 20) + 1, xs=1 << 21), UNSUPPORTED),
])
def test_bwd_refusals(bad, want):
    assert bwd(**bad) == want


def ffn8(x=P, xs=64, s=P, wg=P, sg=P, wu=P, su=P, h=P, T=8, D=64, F=32, act=1, dt=1):
    return L().gated_ffn8_fwd(x, xs, s, wg, sg, wu, su, h, T, D, F, act, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(s=None), INVALID), (dict(wg=None), INVALID), (dict(sg=None), INVALID),
    (dict(wu=None), INVALID), (dict(su=None), INVALID), (dict(h=None), INVALID), (dict(s=ODD), INVALID),
    (dict(sg=ODD), INVALID), (dict(su=ODD), INVALID), (dict(h=ODD), INVALID), (dict(xs=63), INVALID),
    (dict(dt=0), INVALID), (dict(dt=3), INVALID), (dict(act=4), INVALID), (dict(T=0), OK), (dict(T=-1), INVALID),
    (dict(F=1 << 21), UNSUPPORTED),
])
def test_ffn8_refusals(bad, want):
    assert ffn8(**bad) == want


def w4(x=P, xs=64, w=P, s=P, z=None, y=P, R=2, D=64, F=32, group=32, dt=1):
    return L().linear_w4_fwd(x, xs, w, s, z, y, R, D, F, group, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
    (dict(x=ODD), INVALID), (dict(w=ctypes.c_void_p(0x1002)), INVALID), (dict(s=ODD), INVALID), (dict(z=ODD), INVALID),
    (dict(y=ODD), INVALID), (dict(D=60), INVALID), (dict(xs=63), INVALID), (dict(group=16), INVALID),
    (dict(group=256), INVALID), (dict(dt=3), INVALID), (dict(R=-1), INVALID), (dict(F=0), INVALID), (dict(R=0), OK),
    (dict(D=1 << 21, xs=1 << 21), UNSUPPORTED), (dict(R=1 << 31), UNSUPPORTED), (dict(R=1 << 23), UNSUPPORTED),
])
def test_w4_refusals(bad, want):
    assert w4(**bad) == want


def gated_w4(wg=P, sg=P, zg=None, wu=P, su=P, zu=None, h=P, act=1, R=2, **more):
    a = dict(x=P, xs=64, D=64, F=32, group=32, dt=1) | more
    return L().gated_ffn_w4_fwd(a["x"], a["xs"], wg, sg, zg, wu, su, zu, h, R, a["D"], a["F"], a["group"], act, a["dt"], None)


@pytest.mark.parametrize("bad,want", [
    (dict(wg=None), INVALID), (dict(sg=None), INVALID), (dict(wu=None), INVALID), (dict(su=None), INVALID),
    (dict(h=None), INVALID), (dict(zg=P), INVALID), (dict(zu=P), INVALID), (dict(wu=ODD), INVALID), (dict(su=ODD), INVALID),
    (dict(act=4), INVALID), (dict(act=4, R=0), INVALID), (dict(R=0), OK), (dict(D=4, xs=4), INVALID), (dict(x=None), INVALID),
])
def test_gated_w4_refusals(bad, want):
    assert gated_w4(**bad) == want


def nq(x=P, res=P, w=P, r=P, q=P, s=P, R=4, D=64, eps=1e-6, dt=1):
    return L().norm_quant_fwd(x, res, w, r, q, s, R, D, eps, dt, None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(res=None), INVALID), (dict(x=ODD), INVALID), (dict(res=ODD), INVALID), (dict(r=ODD), INVALID),
    (dict(s=ctypes.c_void_p(0x1002)), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(D=0), INVALID), (dict(R=-1), INVALID), (dict(dt=3), INVALID), (dict(D=32769), UNSUPPORTED),
    (dict(R=1 << 31), UNSUPPORTED), (dict(R=1 << 28), UNSUPPORTED), (dict(R=0), OK),
])
def test_norm_quant_refusals(bad, want):
    assert nq(**bad) == want


def test_size_queries():
    out = ctypes.c_size_t()
    q = L().gated_ffn_saved_size
    assert q(8, 32, None) == INVALID and q(-1, 32, ctypes.byref(out)) == INVALID and q(8, 0, ctypes.byref(out)) == INVALID
    assert q(1 << 31, 32, ctypes.byref(out)) == UNSUPPORTED
    assert q(7, 33, ctypes.byref(out)) == OK and out.value == 7 * 2 * 36 * 4
    assert q(0, 33, ctypes.byref(out)) == OK and out.value == 0
    q = L().gated_ffn_bwd_workspace_size
    assert q(8, 64, 32, 1, None) == INVALID and q(8, 64, 32, 3, ctypes.byref(out)) == INVALID
    assert q(8, 1 << 21, 32, 1, ctypes.byref(out)) == UNSUPPORTED
    for dt in (0, 1, 2):
        assert q(8, 64, 32, dt, ctypes.byref(out)) == OK and out.value > 0
        assert q(0, 64, 32, dt, ctypes.byref(out)) == OK


def test_binding_checks_before_the_library():
    x, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        ffn.gated_ffn_fwd(x, w, w)
    with pytest.raises(TypeError):
        ffn.gated_ffn_fwd(x.double(), w, w)
    with pytest.raises(ValueError):
        ffn.gated_ffn_fwd(x[:, :32], w, w)
    with pytest.raises(ValueError):
        ffn._act("relu")
    with pytest.raises(ValueError):
        ffn.linear_w4_fwd(x, torch.zeros(32, 32, dtype=torch.uint8), w[:, :1], group=48)
    with pytest.raises(ValueError):
        ffn.linear_w4_fwd(x[:, :60], torch.zeros(32, 30, dtype=torch.uint8), w[:, :1])
    with pytest.raises(TypeError):
        ffn.gated_ffn8_fwd(x, None, w, None, w, None, dtype=torch.float32)
    with pytest.raises(ValueError):
        ffn.norm_quant_fwd(x, w[0])
    with pytest.raises(ValueError):
        ffn.quantize_w4(torch.zeros(4, 60))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,D", [(32, 64), (64, 72), (128, 40)])
def test_quantized_weights_are_near(zeros, group, D):
    """A weight is off by at most half a step, and by what its scale and zero
    point (float32 here) lose: less than a hundredth of one.  Without zero points
    a step is a seventh of the group's largest value."""
    g = torch.Generator().manual_seed(D)
    w = torch.randn(5, D, generator=g) + 0.5
    w[1] = 0.0
    codes, scales, zero = ffn.quantize_w4(w, group, zeros)
    back = of.weights_w4(codes, scales, zero, group)
    step = scales.double()[:, torch.arange(D) // group]
    assert ((back - w.double()).abs() <= step * 0.51).all()
    assert (back[1] == 0).all()


def test_quantized_rows_are_near():
    w = torch.randn(5, 40, generator=torch.Generator().manual_seed(0))
    w[2] = 0.0
    q, s = ffn.quantize_rows(w)
    off = (q.double() * s.double()[:, None] - w.double()).abs()
    # half a step of e4m3, 2^-4 of the value, or 2^-10 below its smallest normal number
    assert (off <= w.double().abs() * 2 ** -4 * 1.001 + s.double()[:, None] * 2 ** -10).all()


@pytest.mark.parametrize("act", sorted(ffn.ACTS))
def test_definitions_differentiate(act):
    """autograd through the definition against central differences: a step of
    1e-6 leaves about 1e-10 of rounding and 1e-12 of curvature."""
    g = torch.Generator().manual_seed(4)
    leaves = [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True) for s in ((5, 6), (7, 6), (7, 6))]
    fn = lambda: (of.gated_ffn(*leaves, act)[0] ** 2).sum()
    grads = dict(zip(map(id, leaves), torch.autograd.grad(fn(), leaves)))
    with torch.no_grad():
        for t, i, d in _differences(fn, leaves):
            assert abs(grads[id(t)].view(-1)[i].item() - d) <= 1e-6 * (1 + abs(d))
