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


LEAD = {torch.bfloat16: 128, torch.float16: 1024, torch.float32: 0}


def in_norm(t, zero):
    """What a result may be off by, relative to its norm, before it is rounded: a sum of
    n values x (lead + code) has roundings of 2^-24 of its partial sums, about
    (lead + 16) sqrt(n) of x, as the result is about 4 sqrt(n) of x (codes
    around their zero point); 8 of them count for the additions of a group, the
    correction and the sum of the groups."""
    high = LEAD[t] + 16 + (8.0 if zero is None else zero.abs().max().item())
    return high / 4 * 8 * 2.0 ** -24


def off(y, want):
    return ((y.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("t", DTYPES, ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [(1, 4096, 64), (1, 10240, 300), (4, 4104, 33), (7, 1000, 199), (17, 10280, 50), (40, 20000, 24), (70, 33000, 24),
                                  (1, 4104, 8200), (4, 10280, 6200), (16, 10280, 8200), (16, 4104, 6150),
                                  (33, 4104, 6150), (64, 10280, 6150), (130, 4104, 4100)], ids=str)
def test_in_norm(size, group, t):
    """Long rows, whose scales take several turns, in blocks of both sizes: one value
    left out of 33 000 changes a result by 5e-3 of its norm."""
    R, D, F = size
    zeros = (R + group // 32) % 2 == 0
    say("4 bits in norm", size, group, t, zeros)
    codes, scales, zero = weights4(F, D, group, zeros, t, 2 * R + 1)
    x = torch.randn(R, D, generator=gen(5), device=DEV).to(t)
    want = x.double() @ of.weights_w4(codes, scales, zero, group).T
    assert off(ffn.linear_w4_fwd(x, codes, scales, zero, group=group), want) <= half(t) + in_norm(t, zero)


@pytest.mark.parametrize("t", DTYPES, ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [(1, 4104, 64), (4, 10280, 33), (7, 4104, 70), (30, 10280, 40), (64, 4104, 100), (90, 10280, 20),
                                  (1, 10280, 8200), (16, 4104, 8200), (16, 10280, 6150), (32, 10280, 6150),
                                  (64, 4104, 6150)], ids=str)
def test_gated_in_norm(size, group, t):
    """g and u are off as above, h by both (the gates' slopes are at most 1.13, near
    1 for what counts in the norm)."""
    R, D, F = size
    zeros = (F + group // 32) % 2 == 0
    say("gated 4 bits in norm", size, group, t, zeros)
    (cg, sg, zg), (cu, su, zu) = (weights4(F, D, group, zeros, t, s) for s in (2, 3))
    x = torch.randn(R, D, generator=gen(6), device=DEV).to(t)
    want, _, _ = of.gated_ffn(x.double(), of.weights_w4(cg, sg, zg, group), of.weights_w4(cu, su, zu, group), "silu")
    loose = 1.2 * in_norm(t, zg) + in_norm(t, zu) + 2.0 ** -20
    assert off(ffn.gated_ffn_w4_fwd(x, cg, sg, cu, su, zg, zu, group=group), want) <= half(t) + loose


@pytest.mark.parametrize("t", DTYPES, ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("F", [20, 4120, 8200])
def test_values_one_by_one(F, group, t):
    """Rows with a single value, at both ends of pieces, of groups and of what the
    scales' room holds, in the last short piece and at random: the result is one
    weight, whose product is exact but for the zero point's and the scale's (2^-23)
    and the end's rounding."""
    D = 10280
    codes, scales, zero = weights4(F, D, group, True, t, 7)
    w = of.weights_w4(codes, scales, zero, group)
    at = torch.cat((torch.arange(0, D, 512), torch.arange(511, D, 512), torch.arange(128, D, 1024), torch.tensor([31, 32, 63, 64, 127]),
                    torch.arange(10240, D, 7), torch.tensor([D - 1]), torch.randint(0, D, (64,), generator=torch.Generator().manual_seed(1))))
    for rows in (1, 4, 16, 32, 64):
        say("one by one", F, group, t, rows)
        for part in (at.split(rows) if rows > 1 else at[::9].split(1)):
            x = torch.zeros(len(part), D, dtype=t, device=DEV)
            x[torch.arange(len(part)), part] = 1.5
            want = 1.5 * w.T[part.to(DEV)]
            # (zero points are no whole numbers: beside the lead their last digits go)
            room = half(t) * want.abs() * 1.01 + 2.0 ** -22 * (want.abs() + scales.double().amax(1) * (16 + LEAD[t]))
            y = ffn.linear_w4_fwd(x, codes, scales, zero, group=group)
            assert ((y.double() - want).abs() <= room).all(), (part, rows)
