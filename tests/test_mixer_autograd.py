"""The autograd functions of the sequence-mixing operators and of the block,
on the CPU: their products are replaced by elementary ones, and what is looked
at is that a second derivative is refused, never returned as zero."""
import pytest
import torch

from convolution_lowering_amd import mixer, mixer_block


def _conv2d(x, w, layout):
    if layout == "NHWC":
        return torch.einsum("nhwc,ohwc->nhwo", x, w.expand(w.shape[0], 1, 1, -1))
    return torch.einsum("nchw,ochw->nohw", x, w)


def _graph(name, monkeypatch, **more):
    """Leaves and the first output of one function."""
    r = lambda *s: torch.rand(*s, requires_grad=True)
    if name == "conv1d_causal":
        x, w, b = r(5, 3), r(3, 4), r(3)
        monkeypatch.setattr(mixer, "conv1d_causal_fwd", lambda x, w, b, **_: (x * x + b, None))
        monkeypatch.setattr(mixer, "conv1d_causal_bwd",
                            lambda dy, x, w, b, **_: (2 * x * dy, torch.zeros_like(w), dy.sum(0), None))
        return (x, w, b), mixer.conv1d_causal(x, w, b)[0]
    if name == "delta_rule":
        q, k, v, g, beta = r(5, 1, 3), r(5, 1, 3), r(5, 1, 3), r(5, 1), r(5, 1)
        monkeypatch.setattr(mixer, "delta_rule_fwd", lambda q, k, v, g, b, **_: (q * k * v, None, q))
        monkeypatch.setattr(mixer, "delta_rule_bwd", lambda do, q, k, v, g, b, s, **_: (
            do * k * v, do * q * v, do * q * k, torch.zeros_like(g), torch.zeros_like(b), None))
        return (q, k, v, g, beta), mixer.delta_rule(q, k, v, g, beta)[0]
    if name == "branch_norm":
        x, y, w = r(5, 3), r(5, 3), r(3)
        monkeypatch.setattr(mixer, "branch_norm_fwd", lambda x, y, w, g, n, **_: (x + y * y * w, None, y))
        monkeypatch.setattr(mixer, "branch_norm_bwd", lambda dr, dh, x, y, w, g, n, s, **_: (
            dr, 2 * dr * y * w, (dr * y * y).sum(0), None, None))
        return (x, y, w), mixer.branch_norm(x, y, w)[0]
    x, w = r(5, 3), r(4, 3)
    monkeypatch.setattr(mixer_block, "conv2d_fwd", _conv2d)
    return (x, w), mixer_block.project(x, w)


NAMES = ("conv1d_causal", "delta_rule", "branch_norm", "project")


@pytest.mark.parametrize("loss", ["sum", "squares"])
@pytest.mark.parametrize("name", NAMES)
def test_a_second_derivative_is_refused(name, loss, monkeypatch):
    """A gradient penalty beside another term: an error, not the other term's
    gradient alone.  With the sum as the loss the output's own gradient is a
    constant, but the inputs' gradients are not."""
    leaves, y = _graph(name, monkeypatch)
    total = y.sum() if loss == "sum" else (y * y).sum()
    grads = torch.autograd.grad(total, leaves, create_graph=True)
    penalty = sum((g * g).sum() for g in grads)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(penalty + sum((z * z).sum() for z in leaves), leaves)


@pytest.mark.parametrize("name", NAMES)
def test_first_derivatives_are_not(name, monkeypatch):
    """create_graph by itself, and a graph walked twice, give the gradients."""
    leaves, y = _graph(name, monkeypatch)
    a = torch.autograd.grad(y.sum(), leaves, retain_graph=True)
    b = torch.autograd.grad(y.sum(), leaves, create_graph=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and not any(p.requires_grad for p in a)
    y.sum().backward()
    assert all(torch.equal(z.grad, p) for z, p in zip(leaves, a))


def test_a_second_derivative_for_the_state_is_refused(monkeypatch):
    """The state's own gradient does not depend on it, that of q does."""
    monkeypatch.setattr(mixer, "delta_rule_fwd", lambda q, k, v, g, b, *, state, **_: (q * k * v * state, None, q))
    monkeypatch.setattr(mixer, "delta_rule_bwd", lambda do, q, k, v, g, b, s, **_: (
        do * k * v, do * q * v, do * q * k, torch.zeros_like(g), torch.zeros_like(b), do * q * k * v))
    q, k, v, state = (torch.rand(5, 1, 3, requires_grad=True) for _ in range(4))
    g = torch.rand(5, 1)
    y = mixer.delta_rule(q, k, v, g, g, state=state)[0]
    dq, = torch.autograd.grad(y.sum(), (q,), create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad((dq * dq).sum() + (state * state).sum(), (state,))
