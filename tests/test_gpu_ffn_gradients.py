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
