"""The block that runs the sequence-mixing operators together: prompts
continued token by token against the whole sequence at once, and its gradients
against those of the same block in float64."""
import pytest
import torch

from convolution_lowering_amd import mixer
from convolution_lowering_amd.mixer_block import MixerBlock, project
from oracle import mixer as om

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def test_projection_and_its_gradients():
    """Products of bf16 values summed in float32 and rounded once: half a
    step (2^-8), and the rounding of the input gradient's own."""
    g = torch.Generator(device=DEV).manual_seed(0)
    for T, ci, co in ((1, 64, 8), (37, 96, 130), (256, 512, 256)):
        x = torch.randn(T, ci, generator=g, device=DEV).bfloat16().requires_grad_(True)
        w = torch.randn(co, ci, generator=g, device=DEV).bfloat16().requires_grad_(True)
        dy = torch.randn(T, co, generator=g, device=DEV).bfloat16()
        y = project(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        assert _rel(y, x.double() @ w.double().t()) < 2 ** -8
        assert _rel(dx, dy.double() @ w.double()) < 2 ** -8
        assert _rel(dw, dy.double().t() @ x.double()) < 2 ** -8


@torch.no_grad()
def test_tokens_continue_prompts():
    """Prompts, then tokens one by one, give what the whole sequences give.
    Both round to bf16 after each of nine operators (half a step each): 9 of
    those, in norm."""
    block = MixerBlock(width=256, seed=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    lens, more = [70, 1, 129], 6
    xs = [torch.randn(n + more, 256, generator=g, device=DEV).bfloat16() for n in lens]
    norm = lambda x: mixer.branch_norm_fwd(None, x, block.n_next)[0]
    cu = lambda ls: torch.tensor([0] + list(torch.tensor(ls).cumsum(0)), dtype=torch.int32, device=DEV)
    whole = torch.cat(xs)
    _, ref = block(whole, norm(whole), cu([n + more for n in lens]))
    ref = ref.split([n + more for n in lens])
    first = torch.cat([x[:n] for x, n in zip(xs, lens)])
    _, h, states = block(first, norm(first), cu(lens), want_states=True)
    for a, b, n in zip(h.split(lens), ref, lens):
        assert _rel(a, b[:n]) < 9 * 2 ** -8
    pools = block.pools(5)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device=DEV)
    for pool, state in zip(pools, states):
        pool[slots.long()] = state
    for t in range(more):
        tok = torch.stack([x[n + t] for x, n in zip(xs, lens)])
        _, h = block.step(tok, norm(tok), pools, slots)
        assert _rel(h, torch.stack([b[n + t] for b, n in zip(ref, lens)])) < 9 * 2 ** -8


def test_block_gradients():
    """float32 block against the same formulas in float64 (six operators in
    series, each good to 2e-5)."""
    block = MixerBlock(width=96, qk_heads=1, v_heads=2, head=32, dtype=torch.float32, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(90, 96, generator=g, device=DEV)
    h = torch.randn(90, 96, generator=g, device=DEV)
    cu = torch.tensor([0, 20, 90], dtype=torch.int32, device=DEV)
    dx, dh = torch.randn_like(x), torch.randn_like(x)
    params = dict(block.named_parameters())
    out = block(x, h, cu)
    got = torch.autograd.grad(out, list(params.values()), (dx, dh))
    p = {n: v.detach().double().requires_grad_(True) for n, v in params.items()}
    xd, hd = x.double(), h.double()
    gates = hd @ p["w_gates"].t()
    decay = -torch.exp(p["a_log"]) * torch.nn.functional.softplus(gates[:, :2] + p["dt_bias"])
    mixed, _ = om.conv1d_causal(hd @ p["w_qkv"].t(), p["w_conv"], p["b_conv"], cu.tolist(), None, "silu")
    q, k, v = mixed.split((32, 32, 64), -1)
    o, _ = om.delta_rule(q.unflatten(-1, (1, 32)), k.unflatten(-1, (1, 32)), v.unflatten(-1, (2, 32)), decay,
                         torch.sigmoid(gates[:, 2:]), cu.tolist(), None, 32 ** -0.5, True)
    u, _ = om.branch_norm(None, o.reshape(-1, 32), p["n_head"], (hd @ p["w_z"].t()).reshape(-1, 32), None, 1.0, 1e-6, "silu")
    ref = om.branch_norm(xd, u.reshape(90, 64) @ p["w_out"].t(), p["n_post"], p["gate"], p["n_next"], 1.0, 1e-6, "none")
    want = torch.autograd.grad(ref, list(p.values()), (dx.double(), dh.double()))
    for n, a, b in zip(params, got, want):
        assert _rel(a, b) < 1.2e-4, (n, _rel(a, b))
