"""How the attention over a paged cache cuts its work
(csrc/df11_attention_plan.h), built with g++ on its own and checked against
the plan's definition."""

import os
import subprocess

import pytest

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(REPO, "entropy_decoding_df11_amd", "csrc")


@pytest.fixture(scope="module")
def cli(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("attention_plan") / "cli")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", f"-I{CSRC}",
                    os.path.join(REPO, "tests", "cpp", "attention_plan_cli.cpp"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]

    return run


def test_pages(cli):
    """place / page_size up to the largest places and pages, around every multiple that is near them."""
    asked = []
    for size in (1, 2, 3, 5, 7, 16, 24, 40, 48, 127, 128, 255, 256, 1000, 65535, 65536, 65537, (1 << 20) - 1, 1 << 20):
        top = ((1 << 30) + 4096) // size
        for k in {0, 1, 2, top // 3, top // 2, top - 1, top}:
            asked += [(p, size) for p in (k * size - 1, k * size, k * size + 1) if 0 <= p <= (1 << 30) + 8192]
    got = cli([f"P {p} {s}" for p, s in asked])
    assert [g[0] for g in got] == [p // s for p, s in asked]


@pytest.mark.parametrize("units,workgroups", [(1, 512), (7, 512), (511, 512), (512, 512), (513, 512), (100003, 512),
                                              (5, 1), ((1 << 31) - 1, 1023)])
def test_runs_cover_the_units(cli, units, workgroups):
    (line,) = cli([f"R {units} {workgroups}"])
    runs, begins = line[0], line[1:]
    assert 1 <= runs <= workgroups and begins[0] == 0 and begins[-1] == units
    sizes = [b - a for a, b in zip(begins, begins[1:])]
    assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
    some = sorted({u for b in begins for u in (b - 1, b, b + 1) if 0 <= u < units})
    got = cli([f"W {u} {units} {workgroups}" for u in some])
    for u, (w,) in zip(some, got):
        assert begins[w] <= u < begins[w + 1]


@pytest.mark.parametrize("runs", [1, 5, 8, 9, 63, 512, 515])
def test_every_workgroup_has_its_run(cli, runs):
    (got,) = cli([f"X {runs}"])
    assert sorted(got) == list(range(runs))
    for xcd in range(8):  # neighbouring runs on one XCD
        mine = got[xcd::8]
        assert mine == list(range(mine[0], mine[0] + len(mine))) if mine else True


@pytest.mark.parametrize("begin,end,length,n_tokens,capacity", [
    (0, 1, 0, 1, 128), (3, 40, 1000, 64, 4096), (3, 40, 1000, 20, 4096), (0, 5, 100, 5, 96), (0, 5, 100, 5, 0),
    (4, 4, 9, 8, 64), (5, 4, 9, 8, 64), (-1, 4, 9, 8, 64), (0, 4, -1, 8, 64), (8, 12, 1, 8, 64),
    (0, 7, (1 << 31) - 1, 7, 1 << 30), (-2 ** 31, 2 ** 31 - 1, 0, 8, 64), (0, 2 ** 31 - 1, 5, 8, 64),
    (0, 900, 0, 900, 4096), (0, 900, 2500, 1000, 4096), (0, 900, 2500, 1000, 2000), (7, 900, 130, 700, 1 << 20)])
@pytest.mark.parametrize("group,tile_rows", [(1, 16), (4, 16), (7, 32), (1, 256), (5, 128), (64, 16)])
@pytest.mark.parametrize("step,extra", [(128, 0), (128, 4), (1024, 0)])
@pytest.mark.parametrize("masked", [0, 1])
def test_shapes(cli, begin, end, length, n_tokens, capacity, group, tile_rows, step, extra, masked):
    (got,) = cli([f"S {begin} {end} {length} {n_tokens} {capacity} {group} {tile_rows} {step} 3 {masked} {extra}"])
    if begin < 0 or end <= begin or length < 0 or begin >= n_tokens:
        assert got[0] == 0 and got[5] == 0
        return
    tokens, rows = end - begin, min(end, n_tokens) - begin
    places = min(length + tokens, capacity)
    tiles = -(-rows * group // tile_rows)
    assert got[:5] == [tokens, rows, length, places, tiles]
    units = 0
    for tile in range(tiles):
        plain, seen, own, before, first, last = got[6 + 6 * tile:12 + 6 * tile]
        assert plain == min(places, length if masked else length + tile * tile_rows // group + 1)
        row = min((tile * tile_rows + tile_rows - 1) // group, rows - 1)
        assert seen == (places if masked else min(places, length + row + 1))
        assert before == units and first == last == tile
        units += own
        own -= extra
        # enough for what the tile sees, and not many more
        assert own * step >= seen and own >= 1
        # (a table that ends before the sequence does bounds what is seen, not the steps)
        most = -(-(length + row + 1) // step) + 2 + -(-(tile_rows // group + 2) // step)
        assert own <= (max(1, -(-places // step)) if masked else most)
        if masked or capacity <= step:
            assert own == max(1, -(-places // step))
    assert got[5] == 3 * units
