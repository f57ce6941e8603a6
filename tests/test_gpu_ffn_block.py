"""The block's feed-forward half: its operators together, as training, prompts
and single tokens run them."""
import pytest
import torch

from convolution_lowering_amd import mixer
from convolution_lowering_amd.mixer_block import MixerBlock
from oracle import ffn as of
from oracle import mixer as om

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = 2.0 ** -8  # half a step


def _rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def test_a_block_without_is_as_it_was():
    """Neither its parameters nor its results depend on the feed-forward half."""
    plain, more = MixerBlock(width=128, seed=5), MixerBlock(width=128, seed=5, ffn=192)
    mine = dict(more.named_parameters())
    for name, p in plain.named_parameters():
        assert torch.equal(p, mine[name])
    assert len(mine) == len(dict(plain.named_parameters())) + 6
    g = torch.Generator(device=DEV).manual_seed(1)
    x, h = (torch.randn(20, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
    with torch.no_grad():
        qkv, z, decay, b = plain._inputs(h)
        mixed, _ = mixer.conv1d_causal(qkv, plain.w_conv, plain.b_conv)
        q, k, v = plain._heads(mixed)
        o, _ = mixer.delta_rule(q, k, v, decay, b, qk_norm=True)
        want = mixer.branch_norm(x, plain._branch(x, o, z), plain.n_post, plain.gate, plain.n_next)
        assert all(torch.equal(a, c) for a, c in zip(plain(x, h), want))
    with pytest.raises(ValueError):
        plain.quantize()
    with pytest.raises(ValueError):
        more.prompts(x, h)


def test_gradients():
    """float32 block with its feed-forward half against the same formulas in
    float64: ten operators in series, each good to 2e-5."""
    block = MixerBlock(width=96, qk_heads=1, v_heads=2, head=32, dtype=torch.float32, seed=3, ffn=200, act="gelu")
    g = torch.Generator(device=DEV).manual_seed(4)
    x, h, dx, dh = (torch.randn(90, 96, generator=g, device=DEV) for _ in range(4))
    cu = torch.tensor([0, 20, 90], dtype=torch.int32, device=DEV)
    params = dict(block.named_parameters())
    got = torch.autograd.grad(block(x, h, cu), list(params.values()), (dx, dh))
    p = {n: v.detach().double().requires_grad_(True) for n, v in params.items()}
    xd, hd = x.double(), h.double()
    gates = hd @ p["w_gates"].t()
    decay = -torch.exp(p["a_log"]) * torch.nn.functional.softplus(gates[:, :2] + p["dt_bias"])
    mixed, _ = om.conv1d_causal(hd @ p["w_qkv"].t(), p["w_conv"], p["b_conv"], cu.tolist(), None, "silu")
    q, k, v = mixed.split((32, 32, 64), -1)
    o, _ = om.delta_rule(q.unflatten(-1, (1, 32)), k.unflatten(-1, (1, 32)), v.unflatten(-1, (2, 32)), decay,
                         torch.sigmoid(gates[:, 2:]), cu.tolist(), None, 32 ** -0.5, True)
    u, _ = om.branch_norm(None, o.reshape(-1, 32), p["n_head"], (hd @ p["w_z"].t()).reshape(-1, 32), None, 1.0, 1e-6, "silu")
    r, n = om.branch_norm(xd, u.reshape(90, 64) @ p["w_out"].t(), p["n_post"], p["gate"], p["n_next"], 1.0, 1e-6, "none")
    f, _, _ = of.gated_ffn(n, p["w_ffn_gate"], p["w_ffn_up"], "gelu")
    ref = om.branch_norm(r, f @ p["w_ffn_down"].t(), p["n_ffn_post"], p["ffn_gate"], p["n_ffn_next"], 1.0, 1e-6, "none")
    want = torch.autograd.grad(ref, list(p.values()), (dx.double(), dh.double()))
    for n, a, b in zip(params, got, want):
        assert _rel(a, b) < 2e-4, (n, _rel(a, b))


@torch.no_grad()
def test_tokens_continue_prompts():
    """Prompts, then tokens one by one, give what the whole sequences give.  Both
    round to bf16 after each of twelve operators (half a step each): 12 of those, in
    norm."""
    block = MixerBlock(width=256, seed=1, ffn=640)
    g = torch.Generator(device=DEV).manual_seed(2)
    lens, more = [70, 1, 129], 4
    xs = [torch.randn(n + more, 256, generator=g, device=DEV).bfloat16() for n in lens]
    norm = lambda x: mixer.branch_norm_fwd(None, x, block.n_next)[0]
    cu = lambda ls: torch.tensor([0] + list(torch.tensor(ls).cumsum(0)), dtype=torch.int32, device=DEV)
    whole = torch.cat(xs)
    _, ref = block(whole, norm(whole), cu([n + more for n in lens]))
    ref = ref.split([n + more for n in lens])
    first = torch.cat([x[:n] for x, n in zip(xs, lens)])
    _, h, states = block(first, norm(first), cu(lens), want_states=True)
    for a, b, n in zip(h.split(lens), ref, lens):
        assert _rel(a, b[:n]) < 12 * BF16
    pools = block.pools(5)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device=DEV)
    for pool, state in zip(pools, states):
        pool[slots.long()] = state
    for t in range(more):
        tok = torch.stack([x[n + t] for x, n in zip(xs, lens)])
        _, h = block.step(tok, norm(tok), pools, slots)
        assert _rel(h, torch.stack([b[n + t] for b, n in zip(ref, lens)])) < 12 * BF16


@torch.no_grad()
def test_serving_weights():
    """Prompts on 8-bit and tokens on 4-bit weights against the same block on the
    weights that those stand for.  Twelve roundings to bf16 as above; the 8-bit
    rows of h are off by half a step of e4m3 at most, 2^-4 of a value, and their
    products with weights by as much of their norm."""
    block = MixerBlock(width=256, seed=7, ffn=640)
    block.quantize(group=64)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(90, 256, generator=g, device=DEV).bfloat16()
    h = mixer.branch_norm_fwd(None, x, block.n_next)[0]
    cu = torch.tensor([0, 33, 90], dtype=torch.int32, device=DEV)
    kept = {n: p.detach().clone() for n, p in block.named_parameters()}
    got = block.prompts(x, h, cu)
    gate, sg, up, su = block.w8
    block.w_ffn_gate.copy_(gate.float() * sg[:, None])
    block.w_ffn_up.copy_(up.float() * su[:, None])
    want = block(x, h, cu)
    for a, b in zip(got, want):
        assert _rel(a, b) < 12 * BF16 + 2 * 2.0 ** -4
    tokens, ht = x[:5], h[:5]
    pools = block.pools(5)
    for pool in pools:
        pool.normal_(generator=g)
    again = [pool.clone() for pool in pools]
    got = block.step(tokens, ht, pools)
    for name, w4 in zip(("w_ffn_gate", "w_ffn_up", "w_ffn_down"), block.w4):
        dict(block.named_parameters())[name].copy_(of.weights_w4(*w4, 64))
    block.w4 = None
    want = block.step(tokens, ht, again)
    for a, b in zip((*got, *pools), (*want, *again)):
        assert _rel(a, b) < 12 * BF16
    for n, p in block.named_parameters():
        p.copy_(kept[n])


def test_step_of_training_changes_every_parameter():
    block = MixerBlock(width=128, seed=2, ffn=320)
    x = torch.randn(40, 128, generator=torch.Generator(device=DEV).manual_seed(0), device=DEV).bfloat16()
    _, out = block(x, mixer.branch_norm_fwd(None, x, block.n_next)[0])
    (out.float() * torch.linspace(-1, 1, out.numel(), device=DEV).view_as(out)).sum().backward()
    for n, p in block.named_parameters():
        assert p.grad is not None and p.grad.isfinite().all(), n
    for n in ("w_ffn_gate", "w_ffn_up", "w_ffn_down", "n_ffn_post", "n_ffn_next", "ffn_gate"):
        assert dict(block.named_parameters())[n].grad.abs().max() > 0, n
