"""The task walk of kv_q4_attend (which share of the work each block has)
against whole numbers without a limit, at lengths that would take a GPU minutes."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("walk") / "walk.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "q4_walk_host.cpp")])
    L = ctypes.CDLL(so)
    L.walk_per_head.restype = ctypes.c_longlong
    L.walk_find.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p]
    return L


def spans(n, L, G, RT, window):
    """(first visible position, one past the last, tiles) of every query tile."""
    out = []
    for j in range(-(-n * G // RT)):
        first, last = L - n + j * RT // G, L - n + (min(n * G, (j + 1) * RT) - 1) // G
        lo, end = (max(0, first - window + 1) if window else 0), max(last + 1, 0)
        out.append((lo, end, (end - 1) // 128 - lo // 128 + 1 if lo < end else 1))
    return out


SHAPES = [(1, 1, 1, 16), (3, 4096, 6, 32), (5, 2, 4, 16), (300, 1000, 6, 128), (77, 77, 1, 64), (40, 333, 24, 32)]


@pytest.mark.parametrize("n,L,G,RT", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 64, 129, 5000])
def test_tasks_of_a_head(walk, n, L, G, RT, window):
    assert walk.walk_per_head(n, L, G, RT, window) == sum(c for *_, c in spans(n, L, G, RT, window))


@pytest.mark.parametrize("n,G,RT", [(1 << 21, 6, 32), (1 << 20, 16, 16), (3_000_001, 6, 32)])
def test_tasks_of_prompts_of_millions(walk, n, G, RT):
    """Past 2^31 tasks a head: prompts of two million positions with fp32 queries, or with too small a hint."""
    want = sum(c for *_, c in spans(n, n, G, RT, 0))
    assert want > 1 << 31 and walk.walk_per_head(n, n, G, RT, 0) == want


@pytest.mark.parametrize("ph", [1, 7, 4095, 1 << 20, (1 << 31) - 1, (1 << 31) + 5, (1 << 32) + 1, 3 << 33])
def test_a_task_is_found_in_its_head(walk, ph):
    for x in {0, 1, ph - 1, ph, 3 * ph - 1, 3 * ph, 3 * ph + ph // 2, 63 * ph, 64 * ph - 1, *(y for y in ((1 << 32) - 1, 1 << 32) if y < 64 * ph)}:
        g, o = ctypes.c_int(-1), ctypes.c_longlong(-1)
        walk.walk_find(x, ph, ctypes.byref(g), ctypes.byref(o))
        assert (g.value, o.value) == divmod(x, ph), x


LIMIT = (1 << 31) - 1


@pytest.mark.parametrize("n,L,G,RT", SHAPES + [(5, 2, 1, 16), (40, 10, 4, 16), (130, 128, 6, 32), (3, 0, 1, 16), (4096, 4000, 2, 128)])
@pytest.mark.parametrize("window", [0, 1, 7, 4096, 1 << 30, LIMIT - 40, LIMIT - 1, LIMIT])
def test_visible_positions_of_query_tiles(walk, n, L, G, RT, window):
    """Also for rows with more queries than cached positions, whose first places are negative."""
    got = (ctypes.c_int * 4)()
    for j, (lo, end, cnt) in enumerate(spans(n, L, G, RT, window)):
        walk.walk_span(n, L, G, RT, window, j, got)
        if lo < end:
            assert list(got) == [lo, end, lo // 128, cnt]
        else:
            assert got[0] == got[1] and got[3] == 1
        p0, p1 = L - n + j * RT // G, L - n + (min(n * G, (j + 1) * RT) - 1) // G
        for t in range(min(got[2], 1 << 20), min(got[2], 1 << 20) + cnt):
            out_of_sight = 128 * t + 127 > p0 or (window > 0 and 128 * t <= p1 - window)
            assert bool(walk.walk_edge(p0, p1, t, window)) == out_of_sight
