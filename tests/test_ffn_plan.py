"""The sizes of ffn_tiles.py are those that its cases say they are."""
import pytest

from ffn_tiles import CASES, plan


@pytest.mark.parametrize("case", CASES, ids=str)
def test_case_takes_its_tile(case):
    es, kind, (tile, parts), T, D, F = case
    got, splits = plan(es, kind, T, D, F)
    assert (got, splits > 1) == (tile, parts)


def test_every_tile_is_there():
    have = {(es, kind, tile) for es, kind, (tile, _), *_ in CASES}
    want = {(es, kind, tile) for es in (2, 4) for kind in ("fwd", "dx", "dw") for tile in range(5)} | {(1, "fwd", n) for n in range(5)}
    assert have == want - {(2, "dw", 4), (4, "dw", 4)}  # (operands as rows of m have no 32 x 32 tile)
