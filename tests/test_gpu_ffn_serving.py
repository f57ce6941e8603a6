"""Serving with the block's quantized feed-forward weights."""
import pytest
import torch

from convolution_lowering_amd import mixer
from convolution_lowering_amd.mixer_block import MixerBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"


def prepared(seed, n):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, 128, generator=g, device=DEV).bfloat16()
    return x


@torch.no_grad()
def outputs(block, x):
    h = mixer.branch_norm_fwd(None, x, block.n_next)[0]
    return (*block.prompts(x, h), *block.step(x[:3], h[:3], block.pools(3)))


def test_prompts_and_steps_after_training():
    """A block quantized before a training step serves what one quantized after
    it does; so does a step captured before it and replayed after."""
    block, other = (MixerBlock(width=128, seed=3, ffn=192) for _ in range(2))
    x = prepared(1, 40)
    block.quantize()
    before = outputs(block, x)
    pools = block.pools(3)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad():
        h = mixer.branch_norm_fwd(None, x, block.n_next)[0][:3]
    with torch.cuda.graph(graph):
        captured = block.step(x[:3], h, pools)
    for b in (block, other):
        opt = torch.optim.SGD((b.w_ffn_gate, b.w_ffn_up, b.w_ffn_down), lr=50.0)
        _, out = b(x, mixer.branch_norm_fwd(None, x, b.n_next)[0])
        (out.float() * torch.linspace(-1, 1, out.numel(), device=DEV).view_as(out)).sum().backward()
        opt.step()
    other.quantize()
    want = outputs(other, x)
    got = outputs(block, x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not all(torch.equal(a, b) for a, b in zip(got, before))
    for _ in range(3):
        for p in pools:
            p.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want[2:]))


@torch.no_grad()
def test_prompts_keep_the_residual_stream():
    """With a closed feed-forward gate the residual stream of 8-bit prompts is that
    of the block, bit for bit: the branch is added before anything is rounded."""
    block = MixerBlock(width=128, seed=4, ffn=192)
    block.ffn_gate.zero_()
    block.quantize(bits=(8,))
    x = prepared(2, 70)
    h = mixer.branch_norm_fwd(None, x, block.n_next)[0]
    want, got = block(x, h), block.prompts(x, h)
    assert not torch.equal(want[0], x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
