"""Which row and query tile a block of kv_attend_prompt's fp32 kernel has, on the CPU."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def find(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("tiles") / "prompt.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "prompt_host.cpp")])
    L = ctypes.CDLL(so)
    L.tile_from.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 4 + [ctypes.c_longlong, ctypes.c_void_p]

    def call(start, tokens, tile, r, left):
        out = (ctypes.c_int * 3)()
        ok = L.tile_from((ctypes.c_int * len(start))(*start), tokens, len(start) - 1, tile, r, left, out)
        return tuple(out) if ok else None
    return call


@pytest.mark.parametrize("tile", [16, 32, 64])
def test_every_tile_once(find, tile):
    rng = random.Random(tile)
    for rows in (1, 5, 70):
        lens = [rng.choice([0, 0, 1, tile - 1, tile, tile + 1, rng.randrange(0, 500)]) for _ in range(rows)]
        start = [sum(lens[:r]) for r in range(rows + 1)]
        for first in (0, rows // 2):
            want = [(start[r], lens[r], j) for r in range(first, rows) for j in range(-(-lens[r] // tile))]
            assert [find(start, start[-1], tile, first, x) for x in range(len(want))] == want
            assert find(start, start[-1], tile, first, len(want)) is None


def test_rows_over_one_another_stay_inside(find):
    """Starts that go up and down hold the same positions in many rows: more tiles than 2^31. A sum of 32 bits would wrap, and
    the search for the tile pass the last row."""
    T, rows, tile = 1 << 28, 4095, 16
    start = [T * (r % 2) for r in range(rows + 1)]
    each = T // tile
    full = (rows + 1) // 2
    assert full * each > 1 << 32
    for x in (0, each - 1, each, 200 * each + 7, full * each - 1):
        assert find(start, T, tile, 0, x) == (0, T, x % each)
    assert find(start, T, tile, 0, full * each) is None and find(start, T, tile, rows - 1, each) is None
