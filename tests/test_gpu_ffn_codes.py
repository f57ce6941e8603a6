"""4-bit products where the earlier tests' tolerances are wide: large values, long
rows in norm, values one by one."""
import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of
from test_gpu_ffn import DEV, DTYPES, gen, half, say, weights4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 7, 33])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32], ids=str)
def test_large_values(t, group, rows):
    """Finite rows up to the largest number give what their exact products do,
    infinite only where those pass it: a code that stands for zero gives zero."""
    D, F = 264, 20
    say("large values", t, group, rows)
    g = gen(rows + group)
    codes = torch.randint(0, 256, (F, D // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.rand(F, -(-D // group), generator=g, device=DEV) * 2.0 ** -8 + 2.0 ** -10).to(t)
    x = (torch.randn(rows, D, generator=g, device=DEV) * 1e37).to(t)
    w = of.weights_w4(codes, scales, None, group)
    want = x.double() @ w.T
    y = ffn.linear_w4_fwd(x, codes, scales, group=group)
    # rounded once; sums of 128 or 15 times x in float32: 2^-24 of them for each of sqrt(D) additions
    loose = {torch.bfloat16: 144, torch.float32: 16}[t] / 4 * D ** 0.5 * 2.0 ** -24
    assert y.isfinite().all()
    assert (y.double() - want).norm() <= (half(t) + loose) * want.norm()
    codes.fill_(0x88)
    x.fill_(torch.finfo(t).max)
    assert not ffn.linear_w4_fwd(x, codes, scales, group=group).any()
    one = torch.zeros_like(x)
    one[:, 5] = torch.finfo(t).max
    codes.fill_(0xf0)  # 0 and 15 in turn: -8 and 7
    want = one.double() @ of.weights_w4(codes, scales, None, group).T
    y = ffn.linear_w4_fwd(one, codes, scales, group=group).double()
    assert ((y - want).abs() <= want.abs() * (half(t) * 1.01 + 2.0 ** -22)).all()


@pytest.mark.parametrize("rows", [1, 7, 33])
@pytest.mark.parametrize("size", [1e-30, 1e-33])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32], ids=str)
def test_small_values(t, size, rows):
    """Small rows keep their digits, as long as the least of their bf16 parts (2^-16
    of a float32 value) does, times 2^-16, in float32: to 2^-149, in steps of which
    a sum of D products is off by as many at most."""
    D, F, group = 264, 20, 64
    say("small values", t, size, rows)
    codes, scales, zero = weights4(F, D, group, True, t, 3)
    scales = scales / scales  # 1
    x = (torch.randn(rows, D, generator=gen(rows), device=DEV) * size).to(t)
    w = of.weights_w4(codes, scales, zero, group)
    want = x.double() @ w.T
    y = ffn.linear_w4_fwd(x, codes, scales, zero, group=group)
    loose = {torch.bfloat16: 160, torch.float32: 32}[t] / 4 * D ** 0.5 * 2.0 ** -24
    assert (y.double() - want).norm() <= (half(t) + loose) * want.norm() + D * 160 * 2.0 ** -133 * want.numel() ** 0.5
