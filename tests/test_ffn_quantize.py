"""Weights in 4 bits for loading: how far they are from what they stand for."""
import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of


def groups(dtype):
    """Groups around zero, narrow ones around something else, of one value, on one
    side of zero, tiny ones, with an outlier."""
    g = torch.Generator().manual_seed(1)
    rows = [torch.randn(128, generator=g), 3 + 0.02 * torch.randn(128, generator=g), 20 + 0.05 * torch.randn(128, generator=g),
            -1 + 1e-3 * torch.randn(128, generator=g), torch.full((128,), 0.7), torch.zeros(128), torch.full((128,), -5e-5),
            torch.rand(128, generator=g) + 1, 1e-3 * torch.randn(128, generator=g), 2e-6 * torch.randn(128, generator=g),
            torch.cat((torch.randn(127, generator=g) * 0.02, torch.tensor([4.0]))), 1e4 + torch.randn(128, generator=g)]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_half_a_step(zeros, group, dtype):
    """Against the weights as they are (in their dtype): half a step of the group, and
    what the code times scale in float32 loses; a step is no more than a 15th of the
    range (a 7th of the largest value without zero points), and of what the
    zero point's rounding asks for, with two roundings of the scale or its type's
    smallest step."""
    w = groups(dtype)
    codes, scales, zero = ffn.quantize_w4(w, group, zeros)
    assert scales.isfinite().all() and (scales > 0).all() and (zero is None or zero.isfinite().all())
    d = w.double()
    back = of.weights_w4(codes, scales, zero, group)
    step = scales.double()[:, torch.arange(128) // group]
    # float32: the value over the scale and the zero point, each up to |w| / scale + 8, rounded a few times
    loose = (d.abs() + 8 * step) * 2.0 ** -21
    assert ((back - d).abs() <= step * 0.5 + loose).all(), ((back - d).abs() / step).max(1).values
    parts = d.view(len(d), -1, group)
    lo, hi = parts.amin(-1), parts.amax(-1)
    half = torch.finfo(dtype).eps / 2
    most = ((hi - lo) / 15 + (hi + lo).abs() / 15 * half) if zeros else parts.abs().amax(-1) / 7
    same = (hi == lo) if zeros else (parts.abs().amax(-1) == 0)
    smallest = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert (scales.double()[~same] <= (most * (1 + 3 * half) + smallest)[~same]).all()
    if zeros:
        one = same[:, :, None].expand(parts.shape).reshape(d.shape)
        assert torch.equal(back[one], d[one])  # a group of one value is exact
