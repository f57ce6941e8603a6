"""What the feed-forward autograd function asks the library for (on the CPU: the
calls are replaced by the definition)."""
import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of
from test_ffn_boundary import BIG, INVALID, L, ODD, OK, P, WORKSPACE


@pytest.fixture
def calls(monkeypatch):
    """The keywords of each call; results and gradients by the definition."""
    seen = []

    def fwd(x, w_gate, w_up, *, act="silu", save=False):
        seen.append(("fwd", save))
        h, g, u = of.gated_ffn(x, w_gate, w_up, act)
        return h, torch.cat((g, u)) if save else None

    monkeypatch.setattr(ffn, "gated_ffn_fwd", fwd)
    return seen


def leaves(grads=(True, True, True)):
    g = torch.Generator().manual_seed(3)
    return [torch.randn(s, generator=g).requires_grad_(r) for s, r in zip(((5, 6), (7, 6), (7, 6)), grads)]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_saved_without_gradients(mode, calls):
    with mode():
        ffn.gated_ffn(*leaves())
    ffn.gated_ffn(*leaves((False, False, False)))
    assert calls == [("fwd", False)] * 2


@pytest.mark.parametrize("grads", [(True, True, True), (True, False, False), (False, True, False), (False, False, True)])
def test_saved_for_any_gradient(grads, calls):
    h = ffn.gated_ffn(*leaves(grads))
    assert h.requires_grad and calls == [("fwd", True)]
    calls.clear()
    with torch.no_grad(), torch.enable_grad():
        ffn.gated_ffn(*leaves(grads))
    assert calls == [("fwd", True)]


@pytest.mark.parametrize("grads,want", [((True, True, True), (True, True)), ((True, False, False), (True, False)),
                                        ((False, True, True), (False, True)), ((False, False, True), (False, True))])
def test_only_the_gradients_that_are_wanted(grads, want, calls, monkeypatch):
    asked = []

    def bwd(dh, x, w_gate, w_up, saved, *, act="silu", want_dx=True, want_dw=True):
        asked.append((want_dx, want_dw))
        three = [t.detach().requires_grad_(True) for t in (x, w_gate, w_up)]
        with torch.enable_grad():
            dx, dg, du = torch.autograd.grad(of.gated_ffn(*three, act)[0], three, dh)
        return dx if want_dx else None, dg if want_dw else None, du if want_dw else None

    monkeypatch.setattr(ffn, "gated_ffn_bwd", bwd)
    three = leaves(grads)
    for graph in (False, True):
        h = ffn.gated_ffn(*three)
        got = torch.autograd.grad(h.sum(), [t for t in three if t.requires_grad], create_graph=graph)
        ref = torch.autograd.grad(of.gated_ffn(*three, "silu")[0].sum(), [t for t in three if t.requires_grad])
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert asked == [want] * 2


@pytest.mark.parametrize("bad,want", [
    (dict(dx=None, dwg=None, dwu=None), OK), (dict(dwg=None), INVALID), (dict(dwu=None), INVALID), (dict(T=0, dwg=None, dwu=None), OK),
    (dict(dx=None, dwg=None, dwu=None, saved=None), WORKSPACE), (dict(dx=ODD, dwg=None, dwu=None), INVALID),
    (dict(dx=None, dwg=ODD), INVALID), (dict(dx=None, dh=None), INVALID), (dict(dx=None, x=None), INVALID),
])
def test_refusals_of_some_gradients(bad, want):
    a = dict(dh=P, dhs=32, x=P, xs=64, wg=P, wu=P, saved=P, sb=BIG, dx=P, dwg=P, dwu=P, T=8, D=64, F=32, act=1, dt=1, st=None,
             ws=P, nbytes=BIG)
    assert L().gated_ffn_bwd_some(*(a | bad).values()) == want
