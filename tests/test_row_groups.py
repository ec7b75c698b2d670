"""The arithmetic of groups of rows (csrc/row_groups.hpp), compiled for the
host, against whole numbers of any size: offsets that ascend, and offsets that
go back and forth, whose groups have more chunks between them than 32 bits
hold (CPU only)."""

from __future__ import annotations

import random
import subprocess

import pytest

from dense_fp32_tiled_amd import build

PROGRAM = r"""
#include "row_groups.hpp"
#include <stdio.h>
#include <vector>

// stdin: rows, tile rows, places, groups, the offsets; then group numbers, each answered by the smallest and the
// largest of the 64 lanes' counts of chunks before that group, as a wave adds them up
int main() {
    long long rows, tile_rows, places, groups, value, group;
    if (scanf("%lld %lld %lld %lld", &rows, &tile_rows, &places, &groups) != 4) return 1;
    std::vector<int32_t> offsets;
    for (long long i = 0; i <= groups && scanf("%lld", &value) == 1; ++i) offsets.push_back((int32_t)value);
    while (scanf("%lld", &group) == 1) {
        int lane[64];
        for (int c = 0; c < 64; ++c) {
            int64_t own = 0;
            for (long long g = c; g < group; g += 64) own += dft::group_rows(offsets.data(), (int)g, rows).tiles(tile_rows);
            lane[c] = dft::count_at_most(own, places);
        }
        for (int d = 32; d > 0; d /= 2) {
            int then[64];
            for (int c = 0; c < 64; ++c) then[c] = dft::count_at_most((int64_t)lane[c] + lane[c ^ d], places);
            for (int c = 0; c < 64; ++c) lane[c] = then[c];
        }
        int low = lane[0], high = lane[0];
        for (int c = 1; c < 64; ++c) low = lane[c] < low ? lane[c] : low, high = lane[c] > high ? lane[c] : high;
        printf("%d %d\n", low, high);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    work = tmp_path_factory.mktemp("row_groups")
    source, exe = work / "row_groups.cpp", work / "row_groups"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-ftrapv", f"-I{build.CSRC}", str(source), "-o", str(exe)],
                   check=True)

    def run(rows, tile_rows, places, offsets, groups):
        text = " ".join(map(str, [rows, tile_rows, places, len(offsets) - 1, *offsets, *groups]))
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def chunks(offsets, g, rows, tile_rows):
    lo = min(max(offsets[g], 0), rows)
    return -(-(max(lo, min(offsets[g + 1], rows)) - lo) // tile_rows)


def expected(rows, tile_rows, places, offsets, groups):
    before, at = [0], 0
    for g in range(len(offsets) - 1):
        at += chunks(offsets, g, rows, tile_rows)
        before.append(at)
    return [before[g] for g in groups]


def places_for(rows, tile_rows, groups):
    return (rows + groups * (tile_rows - 1)) // tile_rows


@pytest.mark.parametrize("tile_rows", [16, 64])
def test_chunks_before_a_group_of_ascending_offsets(program, tile_rows):
    rng = random.Random(41)
    for groups, rows in [(1, 5), (3, 0), (63, 900), (64, 900), (65, 12345), (1000, 77), (65535, 1 << 23)]:
        offsets = sorted(rng.randint(0, rows) for _ in range(groups + 1))
        places = places_for(rows, tile_rows, groups)
        asked = sorted({0, 1, groups // 2, groups - 1} | {rng.randrange(groups) for _ in range(4)})
        want = expected(rows, tile_rows, places, offsets, asked)
        assert all(w <= places for w in want)
        assert program(rows, tile_rows, places, offsets, asked) == [(w, w) for w in want]


@pytest.mark.parametrize("tile_rows", [16, 64])
def test_chunks_before_a_group_stay_within_their_places(program, tile_rows):
    """Every second group has all rows: from some group on their sum passes 2^31 (the 32-bit sums of the lanes were
    negative there, and the places read in front of the workspace)."""
    rows, groups = 1 << 23, 65535
    offsets = [rows * (g % 2) for g in range(groups + 1)]
    places = places_for(rows, tile_rows, groups)
    asked = [0, 1, 2, 63, 64, 65, 1000, 10000, 40000, 65533, 65534]
    want = expected(rows, tile_rows, places, offsets, asked)
    assert max(want) >= 1 << 31
    assert program(rows, tile_rows, places, offsets, asked) == [(min(w, places),) * 2 for w in want]


def test_offsets_outside_the_rows(program):
    offsets = [-5, 2 ** 31 - 1, -2 ** 31, 7, 3, 900, 2 ** 31 - 1]
    asked = list(range(6))
    want = expected(500, 16, 10 ** 6, offsets, asked)
    assert program(500, 16, 10 ** 6, offsets, asked) == [(w, w) for w in want]
