"""Gradients of the gated product: those that are wanted."""
import pytest
import torch

from convolution_lowering_amd import ffn
from test_gpu_ffn import DEV, DTYPES, gen, inputs, say

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
