"""What the feed-forward autograd function asks the library for (on the CPU: the
calls are replaced by the definition)."""
import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of


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
