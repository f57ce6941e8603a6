"""Sizes at which each tile of the gated products is chosen, for long sums and for
sums in parts."""
import ctypes

import convolution_lowering_amd as cl

# operand bytes, product, (tile, in parts), tokens, width, hidden; tiles as in FfnTileKind: 256 x 128, 256 x 64,
# 128 x 64, 64 x 32, 32 x 32.  What is not here is not chosen.
CASES = [
    (2, "fwd", (0, False), 5000, 776, 776), (2, "fwd", (1, False), 400, 776, 4104), (2, "fwd", (2, False), 5000, 776, 200),
    (2, "fwd", (3, False), 1000, 776, 776), (2, "fwd", (4, False), 3, 776, 72),
    (2, "dx", (0, False), 5000, 1544, 520), (2, "dx", (0, True), 776, 2056, 4104), (2, "dx", (1, False), 5000, 776, 520),
    (2, "dx", (1, True), 136, 3080, 4104), (2, "dx", (2, False), 1304, 1544, 520), (2, "dx", (2, True), 100, 2056, 2600),
    (2, "dx", (3, False), 1000, 1544, 520), (2, "dx", (3, True), 100, 3080, 1800), (2, "dx", (4, False), 1, 64, 520),
    (2, "dx", (4, True), 3, 72, 776),
    (2, "dw", (0, False), 776, 1544, 2600), (2, "dw", (0, True), 4104, 1032, 1800), (2, "dw", (1, False), 776, 1032, 1800),
    (2, "dw", (1, True), 5000, 64, 4104), (2, "dw", (2, False), 776, 200, 4104), (2, "dw", (2, True), 2600, 200, 776),
    (2, "dw", (3, False), 776, 64, 64), (2, "dw", (3, True), 1000, 64, 64),
    (4, "fwd", (0, False), 1000, 520, 8192), (4, "fwd", (1, False), 1000, 520, 4000), (4, "fwd", (2, False), 1000, 520, 1800),
    (4, "fwd", (3, False), 40, 520, 4104), (4, "fwd", (4, False), 3, 520, 72),
    (4, "dx", (0, False), 4096, 4000, 256), (4, "dx", (1, False), 2000, 4000, 256), (4, "dx", (2, False), 1800, 2056, 200),
    (4, "dx", (3, False), 2056, 200, 200), (4, "dx", (3, True), 40, 2056, 2056), (4, "dx", (4, False), 1, 64, 200),
    (4, "dx", (4, True), 3, 72, 520),
    (4, "dw", (0, False), 400, 2000, 4000), (4, "dw", (1, False), 400, 2056, 1800), (4, "dw", (2, False), 400, 1544, 1032),
    (4, "dw", (2, True), 1304, 200, 2056), (4, "dw", (3, False), 400, 64, 64), (4, "dw", (3, True), 520, 64, 64),
    (1, "fwd", (0, False), 5000, 1552, 776), (1, "fwd", (1, False), 400, 1552, 4104), (1, "fwd", (2, False), 5000, 1552, 200),
    (1, "fwd", (3, False), 1000, 1552, 776), (1, "fwd", (4, False), 3, 1552, 72),
]


class _Plan(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("splits", ctypes.c_int)]


def plan(es, kind, T, D, F):
    """(tile, parts) of rows at multiples of 16 bytes."""
    fn = getattr(cl.lib(), "_ZN9convlower8ffn_planEliiibbb")  # convlower::ffn_plan
    fn.restype, fn.argtypes = _Plan, [ctypes.c_int64] + [ctypes.c_int] * 3 + [ctypes.c_bool] * 3
    piece = 128 // es if es > 1 else 64
    both = 2 * -(-F // piece) * piece
    M, N, K = {"fwd": (T, F, D), "dx": (T, D, both), "dw": (both, D, T)}[kind]
    p = fn(M, N, K, es, kind != "fwd", True, kind == "dw")
    return p.tile, p.splits
