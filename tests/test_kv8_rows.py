"""The attention's row arithmetic (csrc/kv8_rows.h) up to the largest call that is accepted, 2^31 - 1 rows, compiled here with
overflow checks."""

import os
import shutil
import subprocess

import pytest

import expert_ffn_decode_gb300 as ffn

CSRC = os.path.join(os.path.dirname(os.path.abspath(ffn.__file__)), "csrc")
MAIN = r"""
#include <cstdio>
#include "kv8_rows.h"
int main() {
  int rows, tile;
  while (std::scanf("%d %d", &rows, &tile) == 2) {
    const int tiles = moe::kv8_tiles(rows, tile), row0 = tiles > 0 ? (tiles - 1) * tile : 0;
    std::printf("%d %d %d\n", tiles, moe::kv8_rows_left(rows, 0, tile), moe::kv8_rows_left(rows, row0, tile));
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or pytest.skip("no g++")
    d = tmp_path_factory.mktemp("kv8_rows")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all", "-I", CSRC, "-o",
                    str(d / "main"), str(d / "main.cpp")], check=True)
    return str(d / "main")


def test_tiles_up_to_the_largest_call(program):
    cases = [(rows, tile) for tile in (8, 16, 130, 240, 254, 256)
             for rows in (0, 1, tile - 1, tile, tile + 1, 12345, 16777215 * 128, 2 ** 31 - 2, 2 ** 31 - 1)]
    r = subprocess.run([program], input="\n".join(f"{a} {b}" for a, b in cases), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for (rows, tile), line in zip(cases, r.stdout.splitlines(), strict=True):
        tiles = -(-rows // tile)
        assert list(map(int, line.split())) == [tiles, min(rows, tile), rows - (tiles - 1) * tile if rows else 0]


def test_kernels_use_it():
    """No sum of a row's number with a tile's rows stands beside it."""
    for name in ("kv8_line.cuh", "kv8_few.cuh", "kv8_many.cu"):
        text = open(os.path.join(CSRC, name)).read()
        for sum_ in ("a.rep + rows - 1", "row0 + 8 *", "row0 + h * half_rows"):
            assert sum_ not in text, (name, sum_)
