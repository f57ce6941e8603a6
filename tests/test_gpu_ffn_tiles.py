"""The gated product and its gradients on each of their tiles, over long sums, in
norm; and sums of which only what lies at the ends of parts and tiles is there.

Norms: a result rounded once is off by half a step of its norm at most, a
gradient by another one for dg and du; a float32 sum of n products, added up
in steps of 32, by 2^-22 sqrt(n / 32) and a few."""
import pytest
import torch

from convolution_lowering_amd import ffn
from ffn_tiles import CASES, plan
from oracle import ffn as of
from test_gpu_ffn import BACK, DEV, DTYPES, gen, half, inputs, rows8, say, tiny

pytestmark = pytest.mark.gpu
TYPES = {2: (torch.bfloat16, torch.float16), 4: (torch.float32,)}


def long_sum(n):
    return (4 + (n / 32) ** 0.5) * 2.0 ** -22


def check(got, want, t, steps, n, what):
    # (below a type's normal numbers half a step is no part of the value but `tiny`: in norm, that for each value)
    off, floor = (got.double() - want).norm().item(), tiny(t) * want.numel() ** 0.5
    assert off <= (steps * half(t) + long_sum(n)) * want.norm().item() + floor, (what, off, want.norm().item())


def each(es):
    return [(t, *c[1:]) for c in CASES if c[0] == es for t in TYPES[es]]


@pytest.mark.parametrize("case", [c for es in (2, 4) for c in each(es) if c[1] == "fwd"], ids=str)
def test_forward(case):
    t, _, tile, T, D, F = case
    say("forward tile", case)
    x, wg, wu = inputs(T, D, F, t)
    h, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    assert torch.equal(h, ffn.gated_ffn_fwd(x, wg, wu)[0])
    want, g, u = of.gated_ffn(x.double(), wg.double(), wu.double(), "silu")
    check(h, want, t, 1, 3 * D, "h")
    pitch = (F + 3) // 4 * 4
    kept = saved.view(torch.float32)[:2 * T * pitch].view(2, T, pitch)[:, :, :F]
    check(kept[0], g, torch.float32, 1, D, "g")
    check(kept[1], u, torch.float32, 1, D, "u")


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == 1], ids=str)
@pytest.mark.parametrize("t", TYPES[2], ids=str)
def test_forward_8_bits(t, case):
    _, _, tile, T, D, F = case
    say("8-bit tile", case, t)
    (x, sx), (wg, sg), (wu, su) = rows8(T, D, 1), rows8(F, D, 2), rows8(F, D, 3)
    sg, su = sg * D ** -0.5, su * D ** -0.5
    h = ffn.gated_ffn8_fwd(x, sx, wg, sg, wu, su, dtype=t)
    want, _, _ = of.gated_ffn(*(z.double() * s.double()[:, None] for z, s in ((x, sx), (wg, sg), (wu, su))), "silu")
    check(h, want, t, 1, 3 * D, "h")


def grads(x, wg, wu, dh):
    """Both passes, and the gradients from the definition."""
    _, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    leaves = [z.double().requires_grad_(True) for z in (x, wg, wu)]
    want = torch.autograd.grad(of.gated_ffn(*leaves, "silu")[0], leaves, dh.double())
    return ffn.gated_ffn_bwd(dh, x, wg, wu, saved), want


@pytest.mark.parametrize("case", [c for es in (2, 4) for c in each(es) if c[1] != "fwd"], ids=str)
def test_gradients(case):
    t, kind, tile, T, D, F = case
    say("gradient tile", case)
    x, wg, wu = inputs(T, D, F, t, 1)
    dh = torch.randn(T, F, generator=gen(2), device=DEV).to(t)
    got, want = grads(x, wg, wu, dh)
    for name, a, b, n in zip(("dx", "dw_gate", "dw_up"), got, want, (2 * F, T, T)):
        check(a, b, t, 2, n + D, name)
    # tokens, or features, at the ends of tiles and parts alone: one left out of n changes the norm by n^-1/2
    es = torch.finfo(t).bits // 8
    piece, (_, parts) = 128 // es, plan(es, kind, T, D, F)
    both = 2 * -(-F // piece) * piece
    n = T if kind == "dw" else F
    tiles = -(-T // piece) if kind == "dw" else both // piece
    ends = [tiles * y // parts * piece for y in range(parts + 1)] + [piece, 2 * piece]
    at = sorted({e % (both // 2) - d if kind == "dx" else e - d for e in ends for d in (0, 1)} & set(range(n)) | {0, n - 1})
    few = torch.zeros_like(dh)
    if kind == "dw":
        few[at] = dh[at]
    else:
        few[:, at] = dh[:, at]
    got, want = grads(x, wg, wu, few)
    for name, a, b in zip(("dx", "dw_gate", "dw_up"), got, want):
        check(a, b, t, 2, 2 * len(at) + D, name + ", ends")


@pytest.mark.parametrize("t", DTYPES, ids=str)
@pytest.mark.parametrize("size", BACK, ids=str)
def test_ragged_gradients(size, t):
    """The sizes of the other tests in norm, and with the last token's, the last
    feature's and a few others' gradient alone."""
    T, D, F = size
    say("ragged gradients", size, t)
    x, wg, wu = inputs(T, D, F, t, 1)
    dh = torch.randn(T, F, generator=gen(2), device=DEV).to(t)
    last, edge = torch.zeros_like(dh), torch.zeros_like(dh)
    last[-1], last[:, -1] = dh[-1], dh[:, -1]
    rows, columns = [torch.arange(0, n, max(1, n // 7), device=DEV) for n in (T, F)]
    edge[rows] = dh[rows]
    edge[:, columns] = dh[:, columns]
    for part in (dh, last, edge):
        got, want = grads(x, wg, wu, part)
        for name, a, b, n in zip(("dx", "dw_gate", "dw_up"), got, want, (2 * F, T, T)):
            check(a, b, t, 2, n + D, name)
