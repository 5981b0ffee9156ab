"""The task walk of kv_q4_attend_tree and kv_attend_prompt's count of blocks on the CPU, and orders between launches that
are read from the sources."""
import ctypes
import os
import random
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mtp_speculative_decoding_step_gb300", "csrc")
LIMIT = (1 << 31) - 1


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("walk") / "tree.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "tree_walk_host.cpp")])
    L = ctypes.CDLL(so)
    L.most_tiles.restype = ctypes.c_longlong
    return L


@pytest.mark.parametrize("n,L", [(1, 1), (1, 128), (1, 129), (16, 4096), (128, 128), (128, 129), (128, 255), (128, 256), (128, 1000), (33, 20), (5, 0),
                                 (128, LIMIT)])
@pytest.mark.parametrize("window", [0, 1, 7, 127, 128, 129, 5000, LIMIT - 1, LIMIT])
def test_tiles_hold_what_nodes_see(walk, n, L, window):
    """All visible positions lie in the tiles; a tile that is no edge is seen whole by every node, whatever the masks and
    depths; edge tiles have numbers of their own, 0 to 3."""
    out = (ctypes.c_int * 4)()
    base = L - n
    for G, RT in ((1, 16), (6, 32), (6, 128)):
        for j in range(-(-n * G // RT)):
            walk.tree_span(n, L, G, RT, window, j, out)
            lo, end, first, count = out
            lowest = max(0, base - window + 1) if window else 0  # of the shallowest node
            assert count >= 1 and first >= 0
            if L > 0:
                assert lo <= max(lowest, 0) and end == L and first == lo // 128 and first + count == (L - 1) // 128 + 1
            numbers = {}
            tiles = sorted({t for t in (first, first + 1, first + 2, max(base, 0) // 128 - 1, max(base, 0) // 128, (max(base, 0) // 128) + 1,
                                        first + count - 1) if first <= t < first + count})
            for t in tiles:
                index = ctypes.c_int()
                edge = walk.tree_edge(n, L, first, t, window, ctypes.byref(index))
                # a position of the tile that the deepest node's window has left, a node, or one past the end
                hidden = 128 * t + 127 >= base or (window > 0 and 128 * t <= L - 1 - window)
                assert bool(edge) == hidden, (t, base)
                if edge and L > n:
                    assert 0 <= index.value < 4 and numbers.setdefault(index.value, t) == t


def test_rows_with_too_many_nodes_have_none(walk):
    start, length, out = (ctypes.c_int * 5)(0, 128, 257, 250, 300), (ctypes.c_int * 4)(500, 500, 9, -4), (ctypes.c_int * 3)()
    got = []
    for r in range(4):
        walk.tree_row(start, length, 290, 10, 16, r, out)
        got.append(tuple(out))
    assert got == [(0, 128, 160), (128, 0, 160), (257, 0, 9), (250, 40, 0)]


def test_blocks_hold_all_units_of_any_rows(walk):
    rng = random.Random(3)
    out = (ctypes.c_int * 2)()
    for _ in range(300):
        rows, G, tile = rng.choice([1, 2, 7, 60]), rng.choice([1, 3, 6]), rng.choice([32, 42, 64, 256])
        lens = [rng.choice([0, 0, 1, 2, tile, tile + 1, rng.randrange(0, 700)]) for _ in range(rows)]
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        arr = (ctypes.c_int * (rows + 1))(*start)
        need = 0
        for r in range(rows):
            walk.prompt_row(arr, start[-1], r, out)
            assert (out[0], out[1]) == (start[r], lens[r])
            need += -(-out[1] * G // tile)
        assert need <= walk.most_tiles(start[-1], rows, G, tile)
    # starts out of order or range stay inside
    arr = (ctypes.c_int * 4)(-7, 10 ** 9, 3, 5)
    got = []
    for r in range(3):
        walk.prompt_row(arr, 20, r, out)
        got.append(tuple(out))
    assert got == [(0, 20), (20, 0), (3, 2)]


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_no_read_only_loads_in_kernels_that_start_before_their_predecessor_ends():
    """As tests/test_q4_order.py: positions, slots, rows and lengths may still be written between a kernel's start and its wait
    for its predecessor."""
    for name in ("kv_rope.cu", "kv_tree.cu", "attn_prompt.cu", "attn_prompt.h", "attn_prompt_tc.cu", "prompt_tiles.h", "tc_attn.cuh"):
        assert not re.findall(r"__ldg|ldg_stream|global\.nc|__restrict__", source(name)), name


def test_kernels_wait_for_their_predecessor_before_they_read():
    for name in ("kv_rope.cu", "kv_tree.cu", "attn_prompt.cu", "attn_prompt_tc.cu"):
        src = source(name)
        for body in re.split(r"__global__", src)[1:]:
            kernel = body[: body.index("\n}\n")]
            wait = kernel.index("pdl_wait()")
            for read in ("a.pos[", "a.slot[", "a.start[", "a.len[", "a.parent[", "a.table[", "find_tile(", "find_unit(", "load4<DT>(", "fetch(0"):
                at = [i.start() for i in re.finditer(re.escape(read), kernel)]
                assert all(i > wait for i in at) or name == "kv_rope.cu" and read in ("a.pos[", "a.slot["), (name, read)


def test_prompt_kernel_takes_tensor_memory_before_a_dependent_kernel_may():
    """A dependent kernel that allocates before its wait would hold what this one's later blocks need."""
    src = source("attn_prompt_tc.cu")
    assert src.index("pdl_wait();") < src.index("tcgen05.alloc") < src.index("pdl_trigger();")


def test_prompt_kernel_waits_with_limits_only():
    """A barrier of some of the warps would keep the others for good where one has left after a wait that ran out."""
    assert not re.findall(r"barrier\.cta|bar\.sync|group_sync|group_any", source("attn_prompt_tc.cu"))
