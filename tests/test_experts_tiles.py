"""The tiles of the experts' products by rows (csrc/plan_tile.h, compiled for the host): of a plan's words as the sort
writes them, and of any others, as a plan of another routing would hold."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scaled_quantize_gemm_gb300", "csrc")
SOURCE = """
#include "plan_tile.h"
extern "C" void tile(const int* d, int t, int num_n, int E, int rows, int half, int* out)
{
    const fp8sq::PlanTile x = fp8sq::plan_tile(d[0], d[1], d[2], d[3], t, num_n, E, rows, half);
    out[0] = x.row0, out[1] = x.end, out[2] = x.nb, out[3] = x.expert;
    for (int rank = 0; rank < 2; ++rank) out[4 + rank] = fp8sq::plan_tile_rows(x, rank);
    out[6] = fp8sq::kTileHalf, out[7] = fp8sq::kTileBox;
}
"""


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan_tile")
    (d / "t.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, str(d / "t.cpp"), "-o", str(d / "t.so")], check=True)
    f = ctypes.CDLL(str(d / "t.so")).tile

    def call(words, t, num_n, E, rows, half=0):
        out = (ctypes.c_int * 8)()
        f((ctypes.c_int * 4)(*words), t, num_n, E, rows, half, out)
        return list(out)
    return call


def _sound(out, num_n, E, rows):
    row0, end, nb, expert, r0, r1, half, box = out
    assert 0 <= row0 <= rows and end <= rows and 0 <= nb < num_n and 0 <= expert < E        # (row0 + 255 below 2^31)
    for rank, r in enumerate((r0, r1)):
        # the bytes that the barrier waits for go by r, the loads by whole boxes of `box` rows
        assert 0 <= r <= half and len(range(0, r, box)) * box == r, out
        # every row that is loaded lies in the buffer
        assert r == 0 or row0 + rank * half + r <= rows, out


@pytest.mark.parametrize("seed", range(4))
def test_any_words(tile, seed):
    rng = random.Random(seed)
    word = lambda: rng.choice([rng.randint(-2 ** 31, 2 ** 31 - 1), rng.randint(-5, 5000), 2 ** 31 - 1, -2 ** 31, 0, -1])     # noqa: E731
    for _ in range(20000):
        num_n, E, rows = rng.randint(1, 60), rng.randint(1, 64), 32 * rng.randint(1, 300)
        out = tile([word() for _ in range(4)], rng.randint(0, 40 * num_n), num_n, E, rows, rng.randint(0, 1))
        _sound(out, num_n, E, rows)


def test_words_of_another_plan(tile):
    """row_of and blocks read as tiles: what a plan made for other sizes gives."""
    rng = random.Random(9)
    for _ in range(5000):
        rows = 32 * rng.randint(1, 200)
        words = ([rng.randint(0, rows - 1) for _ in range(4)] if rng.random() < 0.5 else
                 [rng.randint(0, 31), rng.randint(0, 50), rng.randint(1, 50), rng.randint(1, 32)])
        _sound(tile(words, rng.randint(0, 500), 7, 16, rows), 7, 16, rows)


@pytest.mark.parametrize("num_n", [1, 3, 28])
def test_words_of_its_plan(tile, num_n):
    """Every tile of a plan as the sort writes it: each column tile of each row once, in groups of eight row tiles."""
    rng = random.Random(num_n)
    counts = [rng.choice([0, 1, 31, 32, 33, 128, 129, 255, 256, 257, 3000]) for _ in range(12)]
    rows, tiles, at = sum(-(-c // 32) * 32 for c in counts), [], 0
    want = []
    for e, c in enumerate(counts):
        end = at + -(-c // 32) * 32
        first, m = len(tiles), -(-(end - at) // 256)
        for i in range(m):
            g = i // 8 * 8
            tiles.append([first + g, e << 8 | min(8, m - g), at + 256 * g, end])
        want += [(e, r, nb) for r in range(at, end, 256) for nb in range(num_n)]
        at = end
    seen = []
    for t in range(len(tiles) * num_n):
        row0, end, nb, expert, r0, r1, half, _ = out = tile(tiles[t // num_n], t, num_n, len(counts), rows)
        _sound(out, num_n, len(counts), rows)
        assert r0 + r1 == min(256, end - row0) and r0 == min(128, end - row0)
        seen.append((expert, row0, nb))
    assert sorted(seen) == sorted(want)
