"""The block's copies of its feed-forward weights for serving (on the CPU: no
kernel runs, what would run one is replaced)."""
import copy

import pytest
import torch

from convolution_lowering_amd import ffn, mixer_block
from convolution_lowering_amd.mixer_block import MixerBlock


def block_of(monkeypatch, seed=1, **kw):
    """A block whose prompts and step do nothing but look after the weights."""
    block = MixerBlock(width=64, seed=seed, ffn=96, device="cpu", **kw)
    monkeypatch.setattr(MixerBlock, "_sequences", lambda self, *a: None)
    monkeypatch.setattr(MixerBlock, "_inputs", lambda self, h: (_ for _ in ()).throw(LookupError))
    return block


def serve(block):
    block.prompts(None, None)
    with pytest.raises(LookupError):
        block.step(None, None, None)


def current(block):
    group = block.group
    w8 = (*ffn.quantize_rows(block.w_ffn_gate), *ffn.quantize_rows(block.w_ffn_up))
    w4 = [ffn.quantize_w4(w, group, zeros=True) for w in (block.w_ffn_gate, block.w_ffn_up, block.w_ffn_down)]
    same = lambda a, b: a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return (all(same(a, b) for a, b in zip(block.w8, w8)) and
            all(same(a, b) for p, q in zip(block.w4, w4) for a, b in zip(p, q)))


def trained(block):
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    for p in block.parameters():
        p.grad = torch.ones_like(p)
    opt.step()


def loaded(block):
    block.load_state_dict(MixerBlock(width=64, seed=9, ffn=96, device="cpu").state_dict())


def written(block):
    with torch.no_grad():
        block.w_ffn_down.mul_(2)


def replaced(block):
    block.w_ffn_up = torch.nn.Parameter(block.w_ffn_up.detach() * 3)


def converted(block):
    block.to(torch.float16)


@pytest.mark.parametrize("change", [trained, loaded, written, replaced, converted])
def test_weights_that_changed_are_served(change, monkeypatch):
    block = block_of(monkeypatch)
    block.quantize(32)
    assert current(block)
    change(block)
    assert not current(block)
    serve(block)
    assert current(block)


def test_copies_are_kept_while_weights_are(monkeypatch):
    """Nothing is made again without a change, and the copies stay where they
    are when they are made again."""
    block = block_of(monkeypatch)
    block.quantize(32)
    calls = []
    real = ffn.quantize_w4
    monkeypatch.setattr(ffn, "quantize_w4", lambda *a, **kw: calls.append(1) or real(*a, **kw))
    at = [t.data_ptr() for t in (*block.w8, *(t for w in block.w4 for t in w))]
    serve(block)
    assert not calls
    written(block)
    serve(block)
    assert len(calls) == 3
    assert at == [t.data_ptr() for t in (*block.w8, *(t for w in block.w4 for t in w))]


def test_refused_inside_a_capture(monkeypatch):
    block = block_of(monkeypatch)
    block.quantize(32)
    monkeypatch.setattr(mixer_block, "_capturing", lambda t: True)
    serve(block)
    written(block)
    for call in (lambda: block.prompts(None, None), lambda: block.step(None, None, None)):
        with pytest.raises(RuntimeError):
            call()


def test_other_ways(monkeypatch):
    """Copies taken out stay out; a copied block and one quantized in inference
    mode serve their own weights."""
    block = block_of(monkeypatch)
    block.quantize(32)
    block.w4 = None
    written(block)
    serve_8 = lambda b: b.prompts(None, None)
    serve_8(block)
    assert block.w4 is None and torch.equal(block.w8[1], ffn.quantize_rows(block.w_ffn_gate)[1])
    block.quantize(64)
    other = copy.deepcopy(block)
    written(other)
    serve(other)
    serve(block)
    assert current(other) and current(block)
    with torch.inference_mode():
        block.quantize(32)
        serve(block)
    written(block)
    serve(block)
    assert current(block)


def test_a_refused_call_changes_nothing(monkeypatch):
    """A group that there is not, and widths that 4 bits do not take, leave the
    copies and their group as they were."""
    block = block_of(monkeypatch)
    block.quantize(32)
    with pytest.raises(ValueError):
        block.quantize(48)
    assert block.group == 32 and current(block)
    serve(block)
    odd = MixerBlock(width=64, ffn=97, device="cpu")
    with pytest.raises(ValueError):
        odd.quantize(32)
    assert odd.w8 is None and odd.w4 is None


def test_only_the_copies_asked_for(monkeypatch):
    """8 bits alone, at any width, leave step with the weights themselves; 4 bits
    alone leave no prompts."""
    block = block_of(monkeypatch)
    block.quantize(bits=(8,))
    assert block.w8 is not None and block.w4 is None
    written(block)
    block.prompts(None, None)
    assert block.w4 is None and torch.equal(block.w8[1], ffn.quantize_rows(block.w_ffn_gate)[1])
    block.quantize(32, bits=(4,))
    assert block.w8 is None and block.w4 is not None
    with pytest.raises(ValueError):
        block.prompts(None, None)
    odd = MixerBlock(width=64, ffn=97, device="cpu")
    odd.quantize(bits=(8,))
    assert odd.w8 is not None
    for bad in ((), (16,), (8, 2)):
        with pytest.raises(ValueError):
            block.quantize(bits=bad)
