"""Gradients of the gated product: those that are wanted."""
import math

import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of
from test_gpu_ffn import DEV, DTYPES, gen, half, inputs, near, say, tiny

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", DTYPES, ids=str)
@pytest.mark.parametrize("size", [(0, 24, 40), (5, 24, 40), (130, 250, 77), (300, 264, 520)], ids=str)
def test_some_gradients(size, t):
    """Each product alone gives what both together do."""
    T, D, F = size
    say("some gradients", size, t)
    x, wg, wu = inputs(T, D, F, t)
    dh = torch.randn(T, F, generator=gen(1), device=DEV).to(t)
    _, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    dx, dg, du = ffn.gated_ffn_bwd(dh, x, wg, wu, saved)
    a, none, none2 = ffn.gated_ffn_bwd(dh, x, wg, wu, saved, want_dw=False)
    assert none is none2 is None and torch.equal(a, dx)
    none, b, c = ffn.gated_ffn_bwd(dh, x, wg, wu, saved, want_dx=False)
    assert none is None and torch.equal(b, dg) and torch.equal(c, du)
    assert ffn.gated_ffn_bwd(dh, x, wg, wu, saved, want_dx=False, want_dw=False) == (None, None, None)


def test_a_frozen_layer():
    x, wg, wu = inputs(12, 40, 24, torch.bfloat16)
    x.requires_grad_(True)
    got, = torch.autograd.grad(ffn.gated_ffn(x, wg, wu).sum(), x)
    wg.requires_grad_(True)
    assert torch.equal(torch.autograd.grad(ffn.gated_ffn(x, wg, wu).sum(), (x, wg))[0], got)


def test_saved_of_another_call():
    """What the forward call did not save, or saved for another number of tokens or
    features, is refused."""
    x, wg, wu = inputs(12, 40, 24, torch.bfloat16)
    dh = torch.zeros(12, 24, dtype=torch.bfloat16, device=DEV)
    h, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    for bad in (ffn.gated_ffn_fwd(x, wg, wu)[1], torch.cat((saved, saved)), saved[:-16],
                ffn.gated_ffn_fwd(x[:11], wg, wu, save=True)[1], saved.view(2, -1), saved.cpu()):
        with pytest.raises(ValueError):
            ffn.gated_ffn_bwd(dh, x, wg, wu, bad)
    with pytest.raises(TypeError):
        ffn.gated_ffn_bwd(dh, x, wg, wu, saved.view(torch.float32))
    ffn.gated_ffn_bwd(dh, x, wg, wu, saved)


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("t", DTYPES, ids=str)
def test_slopes_alone(act, t):
    """The gate's slope by itself, relative to its own size: one product for each
    feature (x = u = 1), so that dw_gate is the slope, rounded to t.

    p = 1 / (1 + e^-v) and q = 1 - p: the exponential is off by 2^-22 |v| of
    itself, which changes p by q times that and q by p times that; instructions
    are good to 2^-20 for results of 16 bits, 2^-21 for float32."""
    z = torch.linspace(-40, 40, 641, device=DEV) if t != torch.float16 else torch.linspace(-9, 9, 289, device=DEV)
    z = z.to(t)[:, None].contiguous()
    one = torch.ones(1, 1, dtype=t, device=DEV)
    wu = torch.ones_like(z)
    _, saved = ffn.gated_ffn_fwd(one, z, wu, act=act, save=True)
    _, dg, _ = ffn.gated_ffn_bwd(torch.ones(1, z.shape[0], dtype=t, device=DEV), one, z, wu, saved, act=act)
    zd = z.double()
    c = 2 * math.sqrt(2 / math.pi)
    v = c * (zd + 0.044715 * zd ** 3) if act == "gelu" else zd
    inner = {"sigmoid": torch.ones_like(zd), "silu": zd, "gelu": c * (zd + 3 * 0.044715 * zd ** 3)}[act]
    p, q = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    fast = 2.0 ** -20 if t != torch.float32 else 2.0 ** -21
    wp, wq = fast + 2.0 ** -22 * v.abs() * q, fast + 2.0 ** -22 * v.abs() * p
    turn, rest = p * q * inner, 0 * p if act == "sigmoid" else p  # the slope is their sum
    tol = (wp + wq + 2.0 ** -21) * turn.abs() + (wp + 2.0 ** -22) * rest
    want = turn + rest
    # below the smallest normal numbers (of float32, in which e^-v is taken) nothing has to be kept
    near(dg, want, tol + half(t) * want.abs() * 1.01 + tiny(t) + 1e-34, "dw_gate")


# sizes of dh, x, w_gate, w_up (fp16 ends at 65504 and, with few digits, at 6e-8)
RANGES = {"large": (200, 2.0 ** -6, 2.0 ** -10, 2.0 ** 12),  # dg about 5e4, past it in many places
          "small": (2e-6, 1.0, 2.0 ** -3, 2.0 ** -6),  # dg and du below the smallest normal number
          "usual": (1.0, 1.0, 2.0 ** -3, 2.0 ** -3)}


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("size", [(40, 64, 96), (33, 77, 130), (300, 256, 2048)], ids=str)
@pytest.mark.parametrize("kind", sorted(RANGES))
def test_gradients_of_g_and_u_outside_the_range_of_fp16(kind, size, act):
    """The gradients of g and u may pass what fp16 holds at either end where dx and
    dW do not.  Each of them and each result is rounded once: half a step, in norm,
    and half of the smallest step of a result.  Results past the range are infinite."""
    T, D, F = size
    say("range", kind, size, act)
    g = gen(5)
    sizes = RANGES[kind]
    dh, x, wg, wu = (((torch.randn(s, generator=g, device=DEV)) * k).half() for s, k in
                     zip(((T, F), (T, D), (F, D), (F, D)), sizes))
    _, saved = ffn.gated_ffn_fwd(x, wg, wu, act=act, save=True)
    got = ffn.gated_ffn_bwd(dh, x, wg, wu, saved, act=act)
    leaves = [z.double().requires_grad_(True) for z in (x, wg, wu)]
    h, gd, ud = of.gated_ffn(*leaves, act)
    inner = torch.autograd.grad(h, (gd, ud), dh.double(), retain_graph=True)
    most = max(z.abs().max().item() for z in inner)
    assert {"large": most > 65504, "small": most < 2.0 ** -14, "usual": 1 < most < 1000}[kind]
    for a, b in zip(got, torch.autograd.grad(h, leaves, dh.double())):
        past, near_it = b.abs() > 65504 * 1.01, (b.abs() > 65504 * 0.99) & (b.abs() <= 65504 * 1.01)
        assert (a[past].double() == b[past].sign() * float("inf")).all()
        a, b = a[~(past | near_it)].double(), b[~(past | near_it)]
        assert (a - b).norm() <= 2 * half(torch.float16) * b.norm() + tiny(torch.float16) * b.numel() ** 0.5


def test_a_token_out_of_range_in_fp16():
    """Tokens whose values are not finite do not count for the range of the others,
    and one with large gradients leaves the others their digits."""
    x, wg, wu = inputs(40, 72, 96, torch.float16)
    dh = torch.randn(40, 96, generator=gen(2), device=DEV).half()
    keep = [i for i in range(40) if i != 7]
    dx = lambda dh, x: ffn.gated_ffn_bwd(dh, x, wg, wu, ffn.gated_ffn_fwd(x, wg, wu, save=True)[1])[0]
    want = dx(dh, x)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[7, 70] = bad
        got = dx(dh, y)
        assert torch.equal(got[keep], want[keep]) and not got[7].isfinite().all()
        e = dh.clone()
        e[7, 3] = bad
        got = dx(e, x)
        assert torch.equal(got[keep], want[keep]) and not got[7].isfinite().all()
    e = dh.clone()
    e[7] = 60000.0
    assert torch.equal(dx(e, x)[keep], want[keep])
    assert not dx(torch.zeros_like(dh), x).any()
