"""kv_tree_plan, kv_q4_attend_tree and kv_q4_tree_commit against their plain
forms. The attention's bounds are those of test_gpu_q4_attend: a tree changes
which positions a query sees, not the arithmetic."""
import math
import random

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import tree_ref
from tests.test_gpu_q4_attend import build, call as call_block

pytestmark = pytest.mark.gpu
BAD = 1 << 9
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


def trees(rng, counts, roots=0.0, chain=0.5):
    out = []
    for n in counts:
        par = [-1 if i == 0 or rng.random() < roots else (i - 1 if rng.random() < chain else rng.randrange(i)) for i in range(n)]
        out.append(par)
    return out


def starts(parents):
    return [sum(len(p) for p in parents[:r]) for r in range(len(parents) + 1)]


def run_plan(parents, length, window=0, extra=0):
    """Positions and masks of packed trees behind `extra` unused entries, with that many after them too."""
    flat = [7] * extra + [x for p in parents for x in p] + [7] * extra
    start = [s + extra for s in starts(parents)]
    pos, mask = torch.full((len(flat),), 99, dtype=torch.int32, device="cuda"), torch.full((len(flat), 4), 99, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_tree_plan(i32(flat), i32(start), i32(length), pos, mask, window=window, status=status)
    if extra:
        assert (pos[:extra] == 99).all() and (pos[-extra:] == 99).all() and (mask[-extra:] == 99).all() and (mask[:extra] == 99).all()
        pos, mask = pos[extra:-extra], mask[extra:-extra]
    return pos.cpu(), mask.cpu(), int(status)


@pytest.mark.parametrize("window", [0, 1, 2, 33, 127, 128, 2 ** 31 - 1])
@pytest.mark.parametrize("seed", range(3))
def test_plans(window, seed):
    rng = random.Random(seed)
    counts = [1, 0, 2, 31, 32, 33, 64, 65, 127, 128, 5, 0]
    parents = trees(rng, counts, 0.05, chain=(0.2, 0.6, 0.98)[seed])
    parents.append(list(range(-1, 127)))        # a chain of 128
    parents.append([-1] * 128)                  # nothing but roots
    length = [len(p) + rng.randrange(0, 5000) for p in parents]
    length[3] = 31                              # no prefix
    pos, mask, status = run_plan(parents, length, window, extra=3)
    want_pos, want_masks, want_status = tree_ref.plan(parents, length, window)
    assert status == want_status == 0 and pos.tolist() == want_pos and torch.equal(mask, tree_ref.words(want_masks))


def test_plans_of_what_is_no_tree():
    parents = [[-1, 0, 2, 2, 3, 1], [-1, 5, 1], [-2, 0], [0], [-1, 0], list(range(-1, 128)), [-1, 0, 1]]
    length = [40, 40, 40, 40, 1, 500, -2 ** 31]
    pos, mask, status = run_plan(parents, length)
    want_pos, want_masks, want_status = tree_ref.plan(parents, length)
    assert status == want_status == BAD and pos.tolist() == want_pos and torch.equal(mask, tree_ref.words(want_masks))


def test_plans_with_starts_out_of_range_stay_inside():
    pos, mask = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros((5, 4), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_tree_plan(i32([-1, 0, 0, -1, 0]), i32([-9, 3, 10 ** 9]), i32([3, 2]), pos, mask, status=status)
    assert pos.tolist() == [0, 1, 1, 0, 1] and int(status) == 0


# ------------------------------------------------------------------ attention

def call(c, masks, pos, scale, window=0, max_q=None, want_lse=True, stream=None, q_dev=None, words=None):
    d = lambda x: None if x is None else (x if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32)).cuda()
    cache = m.kv_q4_cache(d(c["kc"]), d(c["vc"]), d(c["k_exp"]), d(c["v_exp"]))
    q = d(c["q"]) if q_dev is None else q_dev
    T, nq, dh = q.shape
    max_q = max_q or max(1, min(128, max(b - a for a, b in zip(c["start"], c["start"][1:]))))
    out = torch.full((T, nq, dh), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, nq), 77.0, device="cuda") if want_lse else None
    ws = torch.full((m.kv_q4_attend_workspace_bytes(cache, nq, max_q, q.dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_attend_tree(cache, q, d(c["table"]), d(c["start"]), d(c["length"]), d(tree_ref.words(masks) if words is None else words), out, ws, max_q,
                        scale=scale, window=window, pos=d(pos) if window else None, lse=lse, status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu(), int(status)


def tolerances(c, masks, pos, scale, window):
    ref, rlse, spread, reach, flat = tree_ref.attend(c["q"].double(), c["kc"], c["vc"], c["table"], c["start"], c["length"], masks, pos, scale, window,
                                                     c["k_exp"], c["v_exp"])
    wide, dh = c["q"].dtype == torch.float32, c["q"].shape[2]
    d = ((2.0 ** -21 if wide else 2.0 ** -16) + dh * 2.0 ** -24) * reach
    rel = 2 * d + 2.0 ** -21 + (2.0 ** -22 if wide else 2.0 ** -11)
    tol = ref.abs() * (2.0 ** -24 if wide else 2.0 ** -8) + rel[..., None] * spread * (1 + 2.0 ** -8) + 1e-30 + 2.0 ** -32 * flat
    return ref, rlse, tol, d + 2.0 ** -20 + rlse.abs() * 2.0 ** -23


def check(c, masks, pos, scale, window=0, **kw):
    out, lse, status = call(c, masks, pos, scale, window, **kw)
    assert status == 0
    ref, rlse, tol, ltol = tolerances(c, masks, pos, scale, window)
    off = (out.double() - ref).abs()
    assert (off <= tol).all(), (float((off / tol).max()), (off > tol).nonzero()[:5])
    empty = rlse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and ((lse.double() - rlse).abs() <= ltol)[~empty].all()
    return out, lse


def planted(counts, kv, nq, nkv, dh, page, dtype, seed, window=0, **kw):
    rng = random.Random(seed)
    parents = trees(rng, counts, **kw)
    c = build(len(counts), counts, kv, nq, nkv, dh, page, dtype, seed)
    pos, masks, status = tree_ref.plan(parents, kv, window)
    assert status == 0
    return c, masks, pos


HEADS = [(4, 2, 64), (8, 2, 128), (24, 4, 256)]


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_small_trees(nq, nkv, dh, dtype, page):
    """Trees of 1 to 9 nodes over lengths around tiles and pages, with and without a prefix."""
    kv = [1, 5, 9, 16, 17, 127, 128, 129, 300, 513, 135]
    n = [1, 5, 9, 2, 3, 4, 1, 5, 9, 3, 9]
    c, masks, pos = planted(n, kv, nq, nkv, dh, page, dtype, dh + page)
    check(c, masks, pos, 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS + [(5, 5, 64), (16, 1, 64), (40, 2, 128), (7, 1, 256)])
@pytest.mark.parametrize("n", [1, 7, 16, 33, 64, 100, 127, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_trees_of_all_sizes(nq, nkv, dh, n, dtype):
    """Up to 128 nodes, whose places may span two tiles; no prefix, short ones, one that ends at a tile's end."""
    c, masks, pos = planted([n, 1, n, n], [n + 200, 37, n, 256 - n % 2], nq, nkv, dh, 32, dtype, n + nq, roots=0.03)
    check(c, masks, pos, 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [1, 2, 64, 129, 130, 5000, 2 ** 31 - 1])
def test_windows(nq, nkv, dh, dtype, window):
    c, masks, pos = planted([3, 60, 1, 128], [600, 333, 129, 300], nq, nkv, dh, 48, dtype, 5, window)
    check(c, masks, pos, 1 / math.sqrt(dh), window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq,nkv,dh", HEADS)
def test_a_chain_is_a_block(nq, nkv, dh, dtype):
    """A tree without branches, by both entry points: within both of their bounds of each other."""
    n, kv = [5, 1, 40], [900, 1300, 77]
    parents = [list(range(-1, k - 1)) for k in n]
    for window in (0, 50):
        pos, masks, _ = tree_ref.plan(parents, kv, window)
        c = build(3, n, kv, nq, nkv, dh, 64, dtype, 3)
        got = call(c, masks, pos, 0.1, window)
        want = call_block(c, 0.1, window)
        assert got[2] == want[2] == 0
        ref, rlse, tol, ltol = tolerances(c, masks, pos, 0.1, window)
        assert ((got[0].double() - want[0].double()).abs() <= 2 * tol).all() and ((got[1].double() - want[1]).abs() <= 2 * ltol).all()


def test_masks_of_any_set():
    """Masks that no tree has: nothing, later nodes, not the node itself, bits past the row's nodes; rows without any position."""
    rng = random.Random(4)
    c = build(4, [40, 3, 2, 0], [500, 3, 2, 50], 8, 2, 128, 16, torch.bfloat16, 31)
    masks = [set(rng.sample(range(40), rng.randrange(0, 40))) for _ in range(40)] + [set(), {2}, {0, 1}] + [set(), set()]
    out, lse = check(c, masks, None, 0.09)
    assert (out[40] == 0).all() and (lse[43:] == -math.inf).all()
    more = [s | {x for x in range(n, 128) if rng.random() < 0.5} for s, n in zip(masks, [40] * 40 + [3] * 3 + [2] * 2)]
    again, lse2, status = call(c, masks, None, 0.09, words=tree_ref.words(more))
    assert status == 0 and torch.equal(again, out) and torch.equal(lse2, lse)


def test_positions_are_held_to_the_row():
    c, masks, pos = planted([6, 9], [400, 300], 8, 2, 128, 16, torch.bfloat16, 6, 70)
    wild = list(pos)
    wild[0], wild[7] = -5, 10 ** 9
    check(c, masks, wild, 0.1, 70)


def test_rows_with_fewer_positions_than_nodes():
    c = build(3, [4, 2, 6], [2, 0, 130], 4, 2, 64, 16, torch.float32, 8)
    masks = [{0}, {0, 1}, {0, 1, 2}, {3}, {0}, {1}] + [set(range(i + 1)) for i in range(6)]
    check(c, masks, None, 0.1)


def test_rows_with_too_many_nodes_are_left_out():
    counts, kv = [3, 129, 5], [200, 400, 90]
    c = build(3, counts, kv, 8, 2, 128, 16, torch.bfloat16, 9)
    parents = trees(random.Random(1), [3]) + [[-1] * 129] + trees(random.Random(2), [5])
    pos, masks, _ = tree_ref.plan(parents, kv)
    out, lse, status = call(c, masks, None, 0.1)
    assert status == BAD and (out[3:132] == 77).all() and (lse[3:132] == 77).all()
    c2 = {**c, "start": [0, 3, 3, 8], "q": torch.cat([c["q"][:3], c["q"][132:]])}
    want, wl, _ = call(c2, masks[:3] + masks[132:], None, 0.1, max_q=128)
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[132:], want[3:]) and torch.equal(lse[132:], wl[3:])


@pytest.mark.parametrize("kv,rows", [(5000, 1), (20000, 2), (3000, 30)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_caches_split_over_many_blocks(kv, rows, dtype):
    lens = [max(12, kv * (i + 1) // rows - 13) for i in range(rows)] if rows > 1 else [kv]
    c, masks, pos = planted([12 if rows < 9 else 3] * rows, lens, 8, 2, 128, 64, dtype, kv)
    check(c, masks, pos, 1 / math.sqrt(128))


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 3, 200])
def test_nan_out_of_sight_stays_out(nq, nkv, dh, dtype, window):
    """NaN in K and V of nodes reaches the nodes below them and no others, in V of the prefix those whose window holds it."""
    L, n = 389, 9
    parent = [-1, 0, 0, 1, 1, 2, 3, 5, 7]
    pos, masks, _ = tree_ref.plan([parent, [-1, 0]], [L, 300], window)
    c = build(2, [n, 2], [L, 300], nq, nkv, dh, 64, dtype, 29)
    clean, _ = check(c, masks, pos, 0.1, window)

    def poison(at, which, head, block):
        c[which][c["table"][0][at // 64], head, at % 64, dh // 2 + block] = 0x7F if at % 2 else 0xFF
    base, G = L - n, nq // nkv
    poison(base + 3, "vc", 0, 1)
    poison(base + 5, "kc", 0, 0)
    if window == 3:
        poison(base - 2, "vc", nkv - 1, 2)  # only depth 0 sees it
    out, _, status = call(c, masks, pos, 0.1, window)
    assert status == 0
    for i in range(n):
        bad = torch.zeros(nq, dh, dtype=torch.bool)
        if 3 in masks[i]:
            bad[:G, 16:32] = True
        if 5 in masks[i]:
            bad[:G] = True
        if window == 3 and pos[i] - (base - 2) < 3:
            bad[nq - G:, 32:48] = True
        assert torch.equal(out[i].isnan(), bad), i
        assert torch.equal(out[i][~bad], clean[i][~bad])
    assert torch.equal(out[n:], clean[n:])


def test_strided_queries_a_small_hint_a_stream_and_a_graph():
    c, masks, pos = planted([5, 40], [300, 90], 8, 2, 128, 16, torch.bfloat16, 24)
    x = torch.zeros(45, 12, 136, dtype=torch.bfloat16, device="cuda")
    view = x[:, 1:9, 3:131]
    view.copy_(c["q"])
    one, _ = check(c, masks, pos, 0.09, q_dev=view)
    two, _ = check(c, masks, pos, 0.09)
    assert torch.equal(one, two)
    check(c, masks, pos, 0.09, max_q=1)
    side = torch.cuda.Stream()
    got, _, _ = call(c, masks, pos, 0.09, want_lse=False, stream=side)
    assert torch.equal(got, two)
    d = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    cache = m.kv_q4_cache(c["kc"].cuda(), c["vc"].cuda(), c["k_exp"].cuda(), c["v_exp"].cuda())
    q, table, start, length, words = c["q"].cuda(), d(c["table"]), d(c["start"]), d(c["length"]), tree_ref.words(masks).cuda()
    out = torch.zeros_like(q)
    ws = torch.empty(m.kv_q4_attend_workspace_bytes(cache, 8, 40, q.dtype), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_q4_attend_tree(cache, q, table, start, length, words, out, ws, 40, scale=0.09)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), two)


@pytest.mark.parametrize("nq,nkv,dh,page", [(24, 4, 256, 64), (8, 2, 128, 64), (4, 2, 64, 16)])
@pytest.mark.parametrize("n", [4, 16, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_repeated_call_gives_the_same_bits(nq, nkv, dh, page, n, dtype):
    c, masks, pos = planted([n, 3, n, 1], [7000, 3001, 3333, 5000], nq, nkv, dh, page, dtype, dh + n)
    first = call(c, masks, pos, 1 / math.sqrt(dh))
    d = lambda x: (x if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32)).cuda()
    cache = m.kv_q4_cache(d(c["kc"]), d(c["vc"]), d(c["k_exp"]), d(c["v_exp"]))
    q, table, start, length, words = d(c["q"]), d(c["table"]), d(c["start"]), d(c["length"]), d(tree_ref.words(masks))
    ws = torch.empty(m.kv_q4_attend_workspace_bytes(cache, nq, n, dtype), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(10):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        m.kv_q4_attend_tree(cache, q, table, start, length, words, out, ws, n, scale=1 / math.sqrt(dh), lse=lse)
        outs.append((out, lse))
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(lse.cpu(), first[1]) and torch.equal(out.cpu(), first[0]), i


# ------------------------------------------------------------------ commit

def commit_case(seed, counts, kv, layers, nkv, dh, page, max_path, match=0.8):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    parents = trees(rng, counts, chain=0.4)
    toks = [[rng.randrange(50) for _ in p] for p in parents]
    choices = []
    for p, t in zip(parents, toks):
        kids = lambda i: [x for x in range(len(p)) if p[x] == i and x > 0]
        choices.append([t[rng.choice(kids(i))] if kids(i) and rng.random() < match else rng.randrange(50) for i in range(len(p))])
    pages = [-(-n // page) for n in kv]
    n_pages = sum(pages) + 2
    perm = torch.randperm(n_pages, generator=g).tolist()
    mp, table, at = max(max(pages), 1), [], 0
    for p in pages:
        table.append(perm[at:at + p] + [-1] * (mp - p))
        at += p
    cache = torch.randint(0, 256, (layers, 2, n_pages, nkv, page, dh * 9 // 16), generator=g, dtype=torch.uint8)
    return parents, toks, choices, table, cache


def run_commit(parents, toks, choices, length, table, cache, max_path, caches=None, with_path=True, stream=None):
    flat = lambda x: i32([y for row in x for y in row])
    R = len(parents)
    dev = cache.cuda()
    cs = m.kv_q4_caches([m.kv_q4_cache(x[0], x[1]) for x in dev])
    o = lambda *s: torch.full(s, 55, dtype=torch.int32, device="cuda")
    n_acc, out_tok, keep, path, status = o(R), o(R, max_path), o(R), o(R, max_path), torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_tree_commit(cs, i32(table), i32(starts(parents)), i32(length), flat(parents), flat(toks), flat(choices), n_acc, out_tok, keep,
                        path=path if with_path else None, status=status, stream=stream)
    torch.cuda.synchronize()
    return n_acc.tolist(), out_tok.tolist(), keep.tolist(), path.tolist(), dev.cpu(), int(status)


def check_commit(parents, toks, choices, length, table, cache, max_path):
    n_acc, out_tok, keep, path, got, status = run_commit(parents, toks, choices, length, table, cache, max_path)
    assert status == 0
    want, page = cache.clone(), cache.shape[4]
    for r, (p, t, k) in enumerate(tree_ref.commit(parents, toks, choices, length, max_path)):
        fill = [-1] * (max_path - len(p))
        assert (n_acc[r], out_tok[r], keep[r], path[r]) == (max(len(p) - 1, 0), t + fill, k, p + fill), r
        base = length[r] - len(parents[r])
        rows = [cache[:, :, table[r][(base + a) // page], :, (base + a) % page].clone() for a in p]
        for place, row in enumerate(rows):
            want[:, :, table[r][(base + place) // page], :, (base + place) % page] = row
    assert torch.equal(got, want)
    return path


@pytest.mark.parametrize("dh,nkv", [(64, 2), (128, 3), (256, 4)])
@pytest.mark.parametrize("layers", [1, 3, 64])
@pytest.mark.parametrize("seed", range(3))
def test_commits(dh, nkv, layers, seed):
    rng = random.Random(seed + layers)
    counts = [1, 16, 2, 33, 128, 7, 0, 64, 16, 16]
    kv = [n + rng.randrange(0, 100) for n in counts]
    kv[3] = 33
    case = commit_case(seed, counts, kv, layers, nkv, dh, (16, 48, 64)[seed], 9, match=(0.8, 0.95, 0.3)[seed])
    check_commit(*case[:3], kv, *case[3:], max_path=(9, 128, 2)[seed])


def test_a_long_path():
    """A chain of 128 accepted whole stays where it is; one of every second node moves together."""
    chain = [list(range(-1, 127)), [-1, 0] + list(range(0, 126))]
    toks = [[5] * 128, [9] + [8] + [5] * 126]
    choices = [[5] * 128] * 2
    kv = [400, 300]
    _, _, _, table, cache = commit_case(3, [128, 128], kv, 2, 2, 128, 32, 128)
    path = check_commit(chain, toks, choices, kv, table, cache, 128)
    assert path[0] == list(range(128)) and path[1][:64] == list(range(0, 128, 2))


def test_commit_without_layers_or_path():
    parents, toks, choices, table, cache = commit_case(5, [9, 3], [50, 40], 1, 2, 64, 16, 9)
    flat = lambda x: i32([y for row in x for y in row])
    o = lambda *s: torch.full(s, 55, dtype=torch.int32, device="cuda")
    n_acc, out_tok, keep = o(2), o(2, 9), o(2)
    m.kv_q4_tree_commit(m.kv_q4_caches([]), None, i32(starts(parents)), i32([50, 40]), flat(parents), flat(toks), flat(choices), n_acc, out_tok, keep)
    for r, (p, t, k) in enumerate(tree_ref.commit(parents, toks, choices, [50, 40], 9)):
        assert (int(n_acc[r]), out_tok[r].tolist(), int(keep[r])) == (len(p) - 1, t + [-1] * (9 - len(p)), k)
    one = run_commit(parents, toks, choices, [50, 40], table, cache, 9)
    two = run_commit(parents, toks, choices, [50, 40], table, cache, 9, with_path=False, stream=torch.cuda.Stream())
    assert one[:3] == two[:3] and torch.equal(one[4], two[4]) and two[3] == [[55] * 9] * 2


def test_commit_faults_move_nothing_of_theirs():
    kv = [60, 60, 10, 200, 129 + 20]
    counts = [9, 9, 12, 5, 129]
    parents, toks, choices, table, cache = commit_case(6, counts, [60, 60, 12, 60, 149], 1, 2, 128, 16, 9)
    parents[0][3] = 3                                  # its own parent: nobody's child
    line = [0, 2, 5]                                   # row 1: path 0, 2, 5, whose last row has no page
    parents[1] = [-1, 0, 0, 0, 0, 2, 0, 0, 0]
    toks[1] = [0, 1, 7, 1, 1, 7, 1, 1, 1]
    choices[1] = [7] * 9
    base = 60 - 9
    bad = [list(t) for t in table]
    assert (base + 1) // 16 == 3 and (base + 5) // 16 == 3
    bad[1][3] = 10 ** 6
    n_acc, out_tok, keep, path, got, status = run_commit(parents, toks, choices, kv, bad, cache, 9)
    assert status == BAD
    want = tree_ref.commit(parents, toks, choices, kv, 9)
    assert path[0][: len(want[0][0])] == want[0][0] and path[1][:4] == line + [-1] and keep[1] == 60 - 9 + 3
    for r in (2, 3, 4):                                # len < n, len past the table, too many nodes
        assert n_acc[r] == 0 and keep[r] == kv[r] and path[r] == [-1] * 9 and out_tok[r] == [-1] * 9
        for p in table[r]:
            if p >= 0:
                assert torch.equal(got[:, :, p], cache[:, :, p])
    for p in table[1]:
        assert torch.equal(got[:, :, p], cache[:, :, p])


def test_commit_in_a_graph():
    parents, toks, choices, table, cache = commit_case(7, [20, 9], [90, 40], 2, 2, 64, 16, 9)
    want = run_commit(parents, toks, choices, [90, 40], table, cache, 9)
    flat = lambda x: i32([y for row in x for y in row])
    dev = cache.cuda()
    cs = m.kv_q4_caches([m.kv_q4_cache(x[0], x[1]) for x in dev])
    o = lambda *s: torch.full(s, 55, dtype=torch.int32, device="cuda")
    args = [i32(table), i32(starts(parents)), i32([90, 40]), flat(parents), flat(toks), flat(choices), o(2), o(2, 9), o(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_q4_tree_commit(cs, *args)
    for _ in range(2):
        dev.copy_(cache)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dev.cpu(), want[4]) and args[7].tolist() == want[1]
