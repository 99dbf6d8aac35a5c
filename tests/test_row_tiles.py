"""How the experts' products cut an expert's rows into tiles, on the host: every
row is in a tile up to the largest count that the calls take, 2^31 - 129."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST_ROWS = 2 ** 31 - 129

# beside every multiple of 32 up to a few tiles, odd sizes, and around where a sum with the tiles' width (2^31 - 255,
# 2^31 - 191) or with their number (2136356790 and 2139127681) passes 31 bits
COUNTS = sorted({*(32 * i + j for i in range(1, 60) for j in (-1, 0, 1)), *(7 ** i for i in range(1, 12)),
                 *(2136356789 + i for i in range(-200, 400)), *(2139127681 + i for i in range(-300, 300)),
                 *(2 ** 31 - i for i in range(129, 700)), *(2 ** i + j for i in range(11, 31) for j in (-1, 0, 1))})


@pytest.mark.parametrize("most", [192, 256])
def test_every_row_is_in_a_tile(tmp_path, most):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "row_tiles")
    # (-fwrapv: a sum that passes 31 bits does here what it does on the GPU)
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fwrapv", "-I",
                           os.path.join(ROOT, "combine_moe_layout_03_gb300", "csrc"),
                           os.path.join(ROOT, "tests", "c", "row_tiles.cpp"), "-o", exe])
    assert max(COUNTS) == MOST_ROWS
    out = subprocess.run([exe, str(most), "0", *map(str, COUNTS)], capture_output=True, text=True, check=True).stdout
    lines = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert lines[0] == (0, 0)
    for rows, (tiles, width) in zip(COUNTS, lines[1:], strict=True):
        assert tiles == -(-rows // most), rows
        assert width == (-(-rows // tiles) + 31) // 32 * 32, rows
        assert 32 <= width <= most and width * tiles >= rows, rows
        assert (tiles - 1) * width < 2 ** 31, rows  # the last tile's first row
