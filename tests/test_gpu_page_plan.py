"""kv_page_plan against a Python stack (whole numbers: equal)."""
import random

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Pool:
    """The plan's state on the device, and one call on it."""

    def __init__(self, table, free, page, max_tokens):
        self.table, self.free, self.page, self.T = dev(table), dev(free), page, max_tokens

    def plan(self, cover, keep, new, stream=None):
        rows = self.table.shape[0]
        out = dict(cover_out=dev([-9] * rows), start=dev([-9] * (rows + 1)), slot=dev([-9] * self.T), pos=dev([-9] * self.T))
        status = dev([0])
        m.kv_page_plan(dev(cover), dev(keep), dev(new), self.table, self.free, out["cover_out"], out["start"],
                       out["slot"], out["pos"], self.page, status=status, stream=stream)
        torch.cuda.synchronize()
        return {**{k: v.tolist() for k, v in out.items()}, "table": self.table.tolist(), "free": self.free.tolist(),
                "fault": int(status.item())}


def check(pool, cover, keep, new):
    ref = q4_ref.plan(cover, keep, new, pool.table.tolist(), pool.free.tolist(), pool.page, pool.T)
    got = pool.plan(cover, keep, new)
    assert got["fault"] == ref["fault"]
    for k in ("cover_out", "start", "slot", "pos"):
        assert got[k] == ref[k], k
    assert got["free"][: len(ref["free"])] == ref["free"]
    for r, n in enumerate(ref["pages"]):
        assert got["table"][r][:n] == ref["table"][r][:n], r
    return got, ref


def start_state(rng, rows, page, max_pages, n_pages, cover):
    perm = list(range(n_pages))
    rng.shuffle(perm)
    table, at = [], 0
    for r in range(rows):
        h = -(-cover[r] // page)
        table.append(perm[at:at + h] + [-1] * (max_pages - h))
        at += h
    return table, perm[at:] + [-5] * at


@pytest.mark.parametrize("rows,page,hi,new_hi,spare", [
    (1, 16, 0, 1, 3), (1, 64, 300, 7, 40), (3, 16, 40, 33, 9), (8, 64, 1000, 4, 100), (33, 48, 500, 100, 200),
    (700, 16, 90, 5, 2000), (1500, 32, 200, 40, 9000), (4096, 16, 64, 3, 9000)])
def test_rounds_of_plans(rows, page, hi, new_hi, spare):
    """Several rounds on one pool: every state, slot and stack entry, including rounds that only trim."""
    rng = random.Random(rows * 7 + page)
    max_pages = -(-(hi + 6 * new_hi) // page) + 1
    cover = [rng.randint(0, hi) for _ in range(rows)]
    n_pages = sum(-(-c // page) for c in cover) + spare
    pool = Pool(*start_state(rng, rows, page, max_pages, n_pages, cover), page, rows * new_hi)
    seen = None
    for turn in range(5):
        keep = [rng.randint(max(0, c - 2 * page), c) for c in cover]
        new = [0 if turn == 3 else rng.randint(0, new_hi) for _ in range(rows)]
        got, ref = check(pool, cover, keep, new)
        again = pool.plan(cover, keep, new)  # the same lengths once more: the same result
        assert again == got
        cover = ref["cover_out"]
        held = [p for r, n in enumerate(ref["pages"]) for p in ref["table"][r][:n]] + ref["free"]
        assert sorted(held) == list(range(n_pages))  # every page is a row's or free, once
        seen = got
    assert seen is not None


def test_an_undone_plan_leaves_the_stack():
    rng = random.Random(5)
    rows, page, max_pages = 9, 16, 12
    cover = [rng.randint(0, 90) for _ in range(rows)]
    n_pages = 90
    pool = Pool(*start_state(rng, rows, page, max_pages, n_pages, cover), page, 400)
    free = pool.free.tolist()
    got, _ = check(pool, cover, cover, [rng.randint(0, 40) for _ in range(rows)])
    check(pool, got["cover_out"], cover, [0] * rows)
    n = n_pages - sum(-(-c // page) for c in cover)
    assert pool.free.tolist()[:n] == free[:n]


def test_the_stack_runs_out_in_row_order():
    page, max_pages = 16, 8
    cover = [16, 0, 40, 16, 0]
    pool = Pool([[0] + [-1] * 7, [-1] * 8, [1, 2, 3] + [-1] * 5, [4] + [-1] * 7, [-1] * 8], [5, 6, 7, 8] + [-1] * 5, page, 300)
    # row 0 takes 1, row 1 two, row 2 gives 2 back (and needs none), row 3 wants 4 of the 3 left, row 4 only 1: refused too
    got, ref = check(pool, cover, [16, 0, 10, 16, 0], [3, 20, 2, 64, 3])
    assert got["fault"] == 1 << 8 and ref["ok"] == [True, True, True, False, False]
    assert got["cover_out"][3:] == [16, 0] and set(got["slot"][25:92]) == {-1}
    check(pool, got["cover_out"], [3, 0, 0, 16, 0], [0, 0, 0, 20, 3])  # trims make room


@pytest.mark.parametrize("cover,keep,new", [
    ([-4, 20], [0, 20], [2, 2]), ([10, 20], [11, 20], [2, 2]), ([10, 20], [-1, 20], [2, 2]), ([10, 20], [10, 20], [-2, 2]),
    ([10, 200], [10, 20], [2, 2]), ([10, 20], [10, 20], [100, 2]), ([10, 20], [10, 20], [2 ** 31 - 1, 2]),
    ([10, 20], [10, 20], [50, 60])])
def test_bad_lengths_are_refused_row_by_row(cover, keep, new):
    pool = Pool([[3] + [-1] * 4, [1, 2] + [-1] * 3], [4, 5, 6, 7, 8, 9, 0, 0, 0, 0], 16, 64)
    if cover[1] == 200:  # claims every page of its table, more than it has: the pool still adds up
        pool = Pool([[3] + [-1] * 4, [1, 2, 0, 4, 5]], [6, 7, 8, 9] + [0] * 6, 16, 64)
    got, ref = check(pool, cover, keep, new)
    assert got["fault"] != 0 and not all(ref["ok"])


def test_more_held_than_there_is_refuses_everything():
    pool = Pool([[0, 1, 2], [0, 1, 2]], [0, 0, 0, 0], 16, 8)
    got = pool.plan([48, 48], [40, 40], [1, 1])
    assert got["fault"] & (1 << 9) and got["cover_out"] == [48, 48] and set(got["slot"]) == {-1}
    assert got["table"] == [[0, 1, 2], [0, 1, 2]] and got["free"] == [0, 0, 0, 0]


def test_entries_that_are_no_pages():
    pool = Pool([[99, -1, -1], [1, -1, -1]], [2, 3, -7, 0, 0, 0], 16, 40)
    # two pages held, so four stack entries: row 1 takes the last of them, page 0
    got = pool.plan([10, 16], [10, 16], [2, 10])
    assert got["fault"] == 1 << 9 and got["slot"][:2] == [-1, -1] and got["slot"][2:12] == list(range(10))
    # then three: row 1's next page would be -7
    got = pool.plan([10, 26], [10, 26], [2, 10])
    assert got["fault"] == 1 << 9 and got["slot"][2:12] == [26 % 16 + i for i in range(6)] + [-1] * 4


def test_captured_into_a_graph_and_on_another_stream():
    rng = random.Random(2)
    cover = [30, 7, 100]
    pool = Pool(*start_state(rng, 3, 16, 12, 40, cover), 16, 30)
    c, k, n = dev(cover), dev([25, 7, 90]), dev([5, 9, 16])
    out = [dev([0] * s) for s in (3, 4, 30, 30)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.kv_page_plan(c, k, n, pool.table, pool.free, *out, 16)
    side.synchronize()
    first = [o.tolist() for o in out]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_page_plan(c, k, n, pool.table, pool.free, *out, 16)
    for o in out:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert [o.tolist() for o in out] == first
