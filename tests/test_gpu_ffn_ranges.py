"""Feed-forward operators where offsets pass 32 bits, on two streams at once, on
other tensors between the replays of a graph, and where inputs hold infinities."""
import pytest
import torch

from convolution_lowering_amd import ffn
from oracle import ffn as of
from test_gpu_ffn import DEV, gated_tolerance, gen, half, inputs, near, say, sums, tiny, w4_tolerance, weights4

pytestmark = pytest.mark.gpu


def some_rows(n):
    return torch.tensor(sorted({0, 1, n // 3, n // 2, (1 << 31) // 8192, n - 2, n - 1} & set(range(n))), device=DEV)


def test_more_than_two_to_the_31_results():
    """300 000 x 8192: the last rows' results, saved products and gradients lie past
    4 and 8 GB."""
    T, D, F = 300_000, 16, 8192
    say("large results", T, D, F)
    x, wg, wu = inputs(T, D, F, torch.bfloat16)
    h, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    at = some_rows(T)
    xd, gd, ud = x[at].double(), wg.double(), wu.double()
    want, g, u = of.gated_ffn(xd, gd, ud, "silu")
    near(h[at], want, gated_tolerance(g, u, sums(xd, gd), sums(xd, ud), "silu", torch.bfloat16), "h")
    dh = torch.zeros_like(h)
    dh[at] = torch.randn(at.numel(), F, generator=gen(1), device=DEV).bfloat16()
    del h
    dx, dg, du = ffn.gated_ffn_bwd(dh, x, wg, wu, saved)
    leaves = [z.requires_grad_(True) for z in (xd, gd, ud)]
    want = torch.autograd.grad(of.gated_ffn(*leaves, "silu")[0], leaves, dh[at].double())
    for got, ref in zip((dx[at], dg, du), want):
        # two roundings to bf16 of half a step each, in norm
        assert (got.double() - ref).norm() <= 2 * half(torch.bfloat16) * ref.norm()
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not dx[rest].any()


def test_more_than_two_to_the_31_normed():
    R, D = 530_000, 4096
    say("large norm", R, D)
    x = torch.empty(R, D, dtype=torch.bfloat16, device=DEV)
    at = some_rows(R)
    x.fill_(1.0)
    x[at] = torch.randn(at.numel(), D, generator=gen(2), device=DEV).bfloat16()
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    q, scale, r = ffn.norm_quant_fwd(x, w, x)
    wq, ws, wr = of.norm_quant(x[at].double(), x[at].double(), w.double(), 1e-6)
    rel = (D / 2 + 12) * 2.0 ** -24
    near(scale[at], ws, rel * ws, "scale")
    near(q[at].float(), wq, (wq.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + 3 * rel * wq.abs(), "q")
    near(r[at], wr, half(torch.bfloat16) * wr.abs(), "r")


def test_more_than_four_gigabytes_of_codes():
    F, D = 1 << 20, 8192 + 40
    say("large codes", F, D)
    g = gen(3)
    codes = torch.randint(0, 256, (F, D // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand(F, -(-D // 128), generator=g, device=DEV).bfloat16()
    x = torch.randn(3, D, generator=g, device=DEV).bfloat16()
    y = ffn.linear_w4_fwd(x, codes, scales)
    at = torch.tensor([0, 17, F // 2, F - 17, F - 1], device=DEV)
    w = of.weights_w4(codes[at], scales[at], None, 128)
    want = x.double() @ w.T
    near(y[:, at], want, w4_tolerance(x.double(), w, scales[at], None, 128, torch.bfloat16) + half(torch.bfloat16) * want.abs() * 1.01, "y")


@pytest.mark.parametrize("size", [(1, 8), (4, 40), (20, 1000), (40, 20000), (70, 33000)], ids=str)
def test_long_rows_of_codes(size):
    """Rows whose scales take several turns of what fits in LDS."""
    R, D = size
    for group in (32, 128):
        for t in (torch.float16, torch.float32):
            say("long codes", R, D, group, t)
            codes, scales, zero = weights4(24, D, group, True, t, 4)
            x = torch.randn(R, D, generator=gen(5), device=DEV).to(t)
            w = of.weights_w4(codes, scales, zero, group)
            want = x.double() @ w.T
            near(ffn.linear_w4_fwd(x, codes, scales, zero, group=group), want,
                 w4_tolerance(x.double(), w, scales, zero, group, t) + half(t) * want.abs() * 1.01 + tiny(t), "y")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [1, 4, 5, 16, 17, 32, 33, 65])
def test_many_features_of_codes(tokens, group, t):
    """As many features as have blocks of half the size, on both sides of each
    number of tokens at which they are shared out another way."""
    D, F = 264 + 8 * (tokens % 3), 6150
    say("many features of codes", tokens, D, F, group, t)
    (cg, sg, zg), (cu, su, zu) = (weights4(F, D, group, tokens % 2 == 0, t, s) for s in (2, 3))
    x = torch.randn(tokens, D, generator=gen(6), device=DEV).to(t)
    xd = x.double()
    wg, wu = of.weights_w4(cg, sg, zg, group), of.weights_w4(cu, su, zu, group)
    eg, eu = w4_tolerance(xd, wg, sg, zg, group, t), w4_tolerance(xd, wu, su, zu, group, t)
    want, g, u = of.gated_ffn(xd, wg, wu, "silu")
    near(ffn.linear_w4_fwd(x, cg, sg, zg, group=group), g, eg + half(t) * g.abs() * 1.01 + tiny(t), "y")
    near(ffn.gated_ffn_w4_fwd(x, cg, sg, cu, su, zg, zu, group=group), want, gated_tolerance(g, u, eg, eu, "silu", t), "h")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_rows_at_any_address(t):
    """x, dh and weights one value past a multiple of 16 bytes, and rows of 4-bit
    products' x that begin at odd ones: the same results as in their place."""
    T, D, F = 70, 136, 264
    x, wg, wu = inputs(T, D, F, t)
    dh = torch.randn(T, F, generator=gen(1), device=DEV).to(t)

    def moved(a):
        flat = torch.empty(a.numel() + 1, dtype=a.dtype, device=DEV)[1:]
        return flat.copy_(a.reshape(-1)).view(a.shape)

    def near_to(a, b):
        # float32 sums in another order, then one rounding
        assert (a.double() - b.double()).norm() <= (2 * half(t) + 300 * 2.0 ** -24) * b.double().norm()

    h, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    near_to(ffn.gated_ffn_fwd(moved(x), moved(wg), moved(wu))[0], h)
    want = ffn.gated_ffn_bwd(dh, x, wg, wu, saved)
    for args in ((moved(dh), x, wg, wu), (dh, moved(x), wg, wu), (dh, x, moved(wg), wu), (dh, x, wg, moved(wu))):
        for a, b in zip(ffn.gated_ffn_bwd(*args, saved), want):
            near_to(a, b)
    codes, scales, zero = weights4(30, D, 32, True, t, 4)
    wide = torch.empty(T, D + 1, dtype=t, device=DEV)
    wide[:, 1:] = x
    for n in (1, 5, 33, 70):
        near_to(ffn.linear_w4_fwd(wide[:n, 1:], codes, scales, zero, group=32), ffn.linear_w4_fwd(x[:n], codes, scales, zero, group=32))
        near_to(ffn.linear_w4_fwd(moved(x[:n]), codes, scales, zero, group=32), ffn.linear_w4_fwd(x[:n], codes, scales, zero, group=32))
    q, s, r = ffn.norm_quant_fwd(moved(x), moved(wg[0]), moved(x))
    q2, s2, r2 = ffn.norm_quant_fwd(x, wg[0], x)
    assert torch.equal(r, r2) and (q.float() - q2.float()).abs().max() <= 32 and (s - s2).abs().max() <= 1e-5 * s2.max()


def test_two_streams_at_once():
    """The same weights in calls that overlap."""
    x, wg, wu = inputs(300, 264, 520, torch.bfloat16)
    dh = torch.randn(300, 520, generator=gen(1), device=DEV).bfloat16()
    codes, scales, _ = ffn.quantize_w4(wg, 64)

    def calls(**on):
        h, saved = ffn.gated_ffn_fwd(x, wg, wu, save=True, **on)
        return (h, *ffn.gated_ffn_bwd(dh, x, wg, wu, saved, **on), ffn.linear_w4_fwd(x, codes, scales, group=64, **on))

    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[calls(stream=s) for s in streams] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for one in pair:
            assert all(torch.equal(a, b) for a, b in zip(one, want))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_keeps_to_its_token(bad):
    """A token with an infinity or a NaN spoils its own results only, and the sums
    over tokens."""
    x, wg, wu = inputs(40, 72, 96, torch.bfloat16)
    clean, saved0 = ffn.gated_ffn_fwd(x, wg, wu, save=True)
    y = x.clone()
    y[7, 70] = bad
    h, saved = ffn.gated_ffn_fwd(y, wg, wu, save=True)
    keep = [i for i in range(40) if i != 7]
    assert torch.equal(h[keep], clean[keep]) and not h[7].isfinite().all()
    dh = torch.randn(40, 96, generator=gen(2), device=DEV).bfloat16()
    a, b = ffn.gated_ffn_bwd(dh, x, wg, wu, saved0)[0], ffn.gated_ffn_bwd(dh, y, wg, wu, saved)[0]
    assert torch.equal(a[keep], b[keep]) and not b[7].isfinite().all()
    # what lies behind the rows and columns that count does not: NaN around the inputs
    wide = torch.full((42, 80), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[1:41, :72] = x
    assert torch.equal(ffn.gated_ffn_fwd(wide[1:41, :72], wg, wu)[0], clean)
    for p, q in zip(ffn.gated_ffn_bwd(dh, wide[1:41, :72], wg, wu, saved0), ffn.gated_ffn_bwd(dh, x, wg, wu, saved0)):
        assert torch.equal(p, q)
    codes, scales, _ = ffn.quantize_w4(wg, 32)
    assert torch.equal(ffn.linear_w4_fwd(wide[1:41, :72], codes, scales, group=32), ffn.linear_w4_fwd(x, codes, scales, group=32))


def test_captured_backward_beside_an_eager_one():
    """A captured training step replayed with eager steps of the same leaves between."""
    x, wg, wu = inputs(50, 64, 96, torch.float32)
    leaves = [z.clone().requires_grad_(True) for z in (x, wg, wu)]

    def step():
        return torch.autograd.grad(ffn.gated_ffn(*leaves).sum(), leaves)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
