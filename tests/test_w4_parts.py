"""The parts of a group's rows that the 4-bit product's tiles work on (csrc/w4_parts.h), on the host: every row in exactly one."""
import ctypes
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_moe_amd", "csrc")


@pytest.fixture(scope="module")
def part_rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cpp").write_text('#include "w4_parts.h"\nextern "C" int part_rows(int l, int t, int p) { return moe::w4_part_rows(l, t, p); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "parts.cpp"), "-o", str(d / "parts.so")], check=True)
    return ctypes.CDLL(str(d / "parts.so")).part_rows


def test_every_row_is_in_one_part(part_rows):
    tile = int(re.search(r"kGroupTile = (\d+)", open(os.path.join(CSRC, "ops_internal.h")).read()).group(1))
    for rows in list(range(1, 3 * tile + 5)) + [10 * tile - 1, 10 * tile, 10 * tile + 129]:
        taken = []
        for first in range(0, rows, tile):  # as moe_sort lists a group's tiles
            for part in (0, 1):
                n = part_rows(rows - first, tile, part)
                assert 0 <= n <= 128
                taken += range(first + 128 * part, first + 128 * part + n)
        assert taken == list(range(rows)), rows


def test_the_kernel_cuts_its_parts_by_it():
    source = open(os.path.join(CSRC, "w4_tile.hip")).read()
    assert source.count("w4_part_rows(") == 3  # both parts' places in the order, and an item's last row
