"""Where the dense products' loads into LDS read (csrc/df11_dense_tiles.h,
composed as df11_dense_kernel composes it), built with g++ on its own: at sizes
that end inside a tile no load reaches past an operand by the lane's own
offset, which is the part that the hardware's range check always covers, and
every element that a tile multiplies comes from its place."""

import os
import re
import subprocess

import pytest

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(REPO, "entropy_decoding_df11_amd", "csrc")


@pytest.fixture(scope="module")
def cli(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("dense_tiles") / "cli")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", f"-I{CSRC}", os.path.join(REPO, "tests", "cpp", "dense_tiles_cli.cpp"),
                    "-o", exe], check=True)

    def run(text):
        return subprocess.run([exe], input=text + "\n", capture_output=True, text=True, check=True).stdout.split("\n")

    return run


def _tile_order_byte(row, col, cols):
    """Byte of W[row][col] in MFMA tile order."""
    panel, r = divmod(row, 64)
    nt, lane16 = divmod(r, 16)
    ks, c = divmod(col, 32)
    return 2 * (((panel * (cols // 32) + ks) * 4 + nt) * 512 + (lane16 + 16 * (c // 8)) * 8 + c % 8)


# few tokens in a tile, one row past a tile, a step and a half along K, one
# k-step, fewer outputs than a tile, rows that are apart, on each other (stride
# 0) and overlapping
SIZES = [(37, 64, 96, 96), (129, 192, 32, 32), (1, 64, 32, 40), (40, 320, 160, 0), (257, 128, 96, 32), (300, 64, 64, 72)]


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("edge", [128, 256])
@pytest.mark.parametrize("tokens,rows,cols,stride", SIZES)
def test_loads_stay_in_the_operands(cli, mode, edge, tokens, rows, cols, stride):
    k_len = rows if mode == 2 else cols
    left_end, right_end = 2 * ((tokens - 1) * stride + k_len), 2 * rows * cols
    outs, n_out = (edge // 2 if mode == 1 else edge), (cols if mode == 2 else rows)
    n_tiles = -(-n_out // outs)
    left, right = {}, {}
    for line in cli(f"T {mode} {edge} {tokens} {rows} {cols} {stride}"):
        f = line.split()
        if not f or f[0] == "E":
            continue
        assert f[0] in "LR", line  # nothing lies partly in a window
        tile, step, lds, at, m = (int(v) for v in f[1:])
        assert 0 <= at and at + 16 <= (left_end if f[0] == "L" else right_end), line
        (left if f[0] == "L" else right)[tile, step, lds] = (at, m)
    for tile in range(-(-tokens // edge) * n_tiles):
        m0, n0 = tile // n_tiles * edge, tile % n_tiles * outs
        for step in range(-(-k_len // 64)):
            # rows of 128 bytes, chunk c at c ^ (row mod 8)
            for r in range(min(edge, tokens - m0)):
                for c in range(8):
                    k = 64 * step + 8 * c
                    if k < k_len:
                        assert left[tile, step, 128 * r + 16 * (c ^ (r % 8))] == (2 * ((m0 + r) * stride + k), 0)
            for b in range(edge // 8):
                for lane in range(64):
                    if mode == 2:  # block b: k-step b / 4 of the outputs, rows 16 (b mod 4)
                        row, col, m = 64 * step + 16 * (b % 4) + lane % 16, n0 + 32 * (b // 4) + 8 * (lane // 16), 0
                    else:
                        half, nb = divmod(b, edge // 16)
                        m = int(mode == 1 and nb % 4 >= 2)
                        out = 16 * (nb // 4 * 2 + nb % 2) if mode == 1 else 16 * nb
                        row, col = n0 + out + lane % 16, 64 * step + 32 * half + 8 * (lane // 16)
                    if row < rows and col < cols:
                        assert right[tile, step, 1024 * b + 16 * lane] == (_tile_order_byte(row, col, cols), m)


def test_offsets_fit_32_bits(cli):
    """The largest strides and widths the products accept."""
    stride = 1 << 22
    assert int(cli(f"O 63 31 {stride}")[0]) == 255 * stride * 2 + 16 * (7 ^ 7)
    panel = (1 << 22) // 32 * 4096
    assert int(cli(f"B 15 1 {panel}")[0]) == 3 * panel + 4096 + 3 * 1024


def test_loads_have_no_scalar_offset():
    """The kernel's one load into LDS passes all of a lane's offset where the
    range check sees it."""
    src = open(os.path.join(CSRC, "df11_dense.hip")).read()
    calls = re.findall(r"buffer_load_lds\(([^;]*);", src)
    assert len(calls) == 1 and re.sub(r"\s", "", calls[0]).endswith(",16,lane_at,0,0,0)")
