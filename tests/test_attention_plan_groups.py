"""The steps that the plan of the attention's work (csrc/df11_attention_plan.h) counts
for the tiles of long prompts, for groups of query heads that do not divide them,
against what each tile sees (the program of test_attention_plan.py)."""

import pytest

from test_attention_plan import cli  # noqa: F401


@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 9, 12, 64])
@pytest.mark.parametrize("tile_rows,step", [(16, 256), (64, 128), (128, 128), (256, 128), (256, 32)])
@pytest.mark.parametrize("tokens,length,n_tokens,capacity", [
    (10000, 0, 10000, 1 << 14), (4001, 130, 4001, 1 << 13), (3000, 2500, 3000, 1 << 13), (3000, 127, 1001, 1 << 13),
    (5000, 500, 5000, 3000), (5000, 5000, 5000, 3000), (257, 1, 257, 1 << 13)])
def test_steps_of_prompts(cli, tokens, length, n_tokens, capacity, group, tile_rows, step):  # noqa: F811
    """At most one more than a tile needs, or a full tile's own more at a sequence's end; all if its pages end before."""
    (got,) = cli([f"S 0 {tokens} {length} {n_tokens} {capacity} {group} {tile_rows} {step} 1 0 2"])
    rows = min(tokens, n_tokens)
    places = min(length + tokens, capacity)
    tiles = -(-rows * group // tile_rows)
    assert got[3] == places and got[4] == tiles
    units = 0
    for tile in range(tiles):
        _, seen, own, before, first, last = got[6 + 6 * tile:12 + 6 * tile]
        row = min((tile * tile_rows + tile_rows - 1) // group, rows - 1)
        assert seen == min(places, length + row + 1)
        assert before == units and first == last == tile
        units += own
        needs = -(-seen // step)
        most = needs + 1 + (tile == tiles - 1) * -(-tile_rows // (step * group))
        if length + tokens > capacity or tiles == 1:
            most = -(-places // step)
        assert needs <= own - 2 <= most
    assert got[5] == units
