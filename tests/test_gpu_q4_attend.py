"""kv_q4_attend against plain 64-bit attention over the same bytes.

Bounds (derived, then fixed): a score is a sum of dh products in fp32 of q
rounded to f16 (bf16 input: exact but for elements far below the largest, 2^-16
of it; fp32: two parts, 2^-22), so it is off by at most
  d = (2^-16 or 2^-21 + dh 2^-24) scale sum |q k|,
a softmax weight by 2 d + 2^-21 of itself and, for bf16, its own f16 rounding
(2^-11; fp32: two parts, 2^-22), an output element by that times sum p |v|, and
finally by its type's half step; lse by d + 2^-20 and its own half step.
Weights are held as 2^(y - m) with the largest at 2^7 at the least, so f16's
smallest spacing of 2^-24 moves each by up to 2^-25, 2^-32 of the largest: an
output element by 2^-32 sum |v|, which shows only where the positions that carry
the weight have v = 0."""
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref

pytestmark = pytest.mark.gpu


def build(rows, q_len, kv_len, nq, nkv, dh, page, dtype, seed, exps=True, q_scale=1.5):
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in kv_len]
    n_pages = sum(pages) + 2
    perm = torch.randperm(n_pages, generator=g).tolist()
    mp = max(max(pages), 1) + 1
    table, at = [], 0
    for p in pages:
        table.append(perm[at:at + p] + [-1] * (mp - p))
        at += p
    kc, vc = (q4_ref.quantize(torch.randn((n_pages * nkv, page, dh), generator=g))[0].reshape(n_pages, nkv, page, -1)
              for _ in range(2))
    # slots past a row's length hold whatever was there: NaN rows
    for r, n in enumerate(kv_len):
        if n % page:
            kc[table[r][n // page], :, n % page:] = 0x7F
            vc[table[r][n // page], :, n % page:] = 0xFF
    T = sum(q_len)
    q = (q_scale * torch.randn((T, nq, dh), generator=g)).to(dtype)
    start = [sum(q_len[:r]) for r in range(rows + 1)]
    ke = torch.tensor([h % 3 - 1 for h in range(nkv)], dtype=torch.int32) if exps else None
    ve = torch.tensor([2 - h % 5 for h in range(nkv)], dtype=torch.int32) if exps else None
    return dict(kc=kc, vc=vc, table=table, start=start, length=list(kv_len), q=q, k_exp=ke, v_exp=ve)


def call(c, scale, window=0, max_q=None, q_dev=None, want_lse=True, stream=None):
    d = lambda x: None if x is None else (x if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32)).cuda()
    cache = m.kv_q4_cache(d(c["kc"]), d(c["vc"]), d(c["k_exp"]), d(c["v_exp"]))
    q = d(c["q"]) if q_dev is None else q_dev
    T, nq, dh = q.shape
    max_q = max_q or max(1, max(b - a for a, b in zip(c["start"], c["start"][1:])))
    out = torch.full((T, nq, dh), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, nq), 77.0, device="cuda") if want_lse else None
    ws = torch.full((m.kv_q4_attend_workspace_bytes(cache, nq, max_q, q.dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_attend(cache, q, d(c["table"]), d(c["start"]), d(c["length"]), out, ws, max_q, scale=scale, window=window,
                   lse=lse, status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu(), int(status)


def check(c, scale, window=0, **kw):
    out, lse, status = call(c, scale, window, **kw)
    assert status == 0
    ref, rlse, spread, reach, flat = q4_ref.attend(c["q"].double(), c["kc"], c["vc"], c["table"], c["start"], c["length"],
                                                   scale, window, c["k_exp"], c["v_exp"])
    wide = c["q"].dtype == torch.float32
    dh = c["q"].shape[2]
    d = ((2.0 ** -21 if wide else 2.0 ** -16) + dh * 2.0 ** -24) * reach
    rel = 2 * d + 2.0 ** -21 + (2.0 ** -22 if wide else 2.0 ** -11)
    tol = ref.abs() * (2.0 ** -24 if wide else 2.0 ** -8) + rel[..., None] * spread * (1 + 2.0 ** -8) + 1e-30 + 2.0 ** -32 * flat
    off = (out.double() - ref).abs()
    assert (off <= tol).all(), (float((off / tol).max()), (off > tol).nonzero()[:5])
    empty = rlse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    ltol = d + 2.0 ** -20 + rlse.abs() * 2.0 ** -23
    assert ((lse.double() - rlse).abs() <= ltol)[~empty].all()
    return out, lse


HEADS = [(4, 2, 64), (8, 2, 128), (24, 4, 256)]


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 48, 64, 128])
def test_short_blocks(nq, nkv, dh, dtype, page):
    """Blocks of 1 to 5 queries; lengths around tiles, pages and their ends."""
    kv = [1, 5, 15, 16, 17, 127, 128, 129, 300, 513]
    q = [1, 5, 1, 2, 3, 4, 1, 5, 4, 3]
    c = build(len(kv), q, kv, nq, nkv, dh, page, dtype, 100 + dh + page)
    check(c, 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS + [(5, 5, 64), (3, 1, 128), (16, 1, 64), (40, 2, 128), (7, 1, 256)])
@pytest.mark.parametrize("n", [1, 2, 3, 6, 11, 17, 33, 70])
def test_blocks_of_all_widths(nq, nkv, dh, n):
    """From one query row per KV head to more than any tile holds."""
    c = build(3, [n, 1, n], [n + 200, 37, n], nq, nkv, dh, 32, torch.bfloat16, n + nq)
    check(c, 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [1, 2, 64, 129, 5000])
def test_windows(nq, nkv, dh, dtype, window):
    c = build(3, [3, 40, 1], [600, 333, 129], nq, nkv, dh, 48, dtype, window)
    check(c, 1 / math.sqrt(dh), window)


def test_rows_that_see_nothing():
    """No cache at all, fewer positions than queries, no queries."""
    c = build(4, [2, 3, 0, 1], [0, 2, 50, 40], 8, 2, 128, 16, torch.bfloat16, 3)
    out, lse = check(c, 0.1)
    assert (out[:3] == 0).all() and (lse[:3] == -math.inf).all() and (out[3:] != 0).any()


@pytest.mark.parametrize("kv,rows", [(5000, 1), (20000, 2), (3000, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_caches_split_over_many_blocks(kv, rows, dtype):
    lens = [max(1, kv * (i + 1) // rows - 13) for i in range(rows)] if rows > 1 else [kv]
    c = build(rows, [2 if rows < 9 else 1] * rows, lens, 8, 2, 128, 64, dtype, kv)
    check(c, 1 / math.sqrt(128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq,nkv,dh", HEADS)
def test_a_prompt_behind_a_prefix(nq, nkv, dh, dtype):
    c = build(2, [150, 77], [700, 77], nq, nkv, dh, 64, dtype, 9)
    check(c, 1 / math.sqrt(dh))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_that_grow_along_the_cache(dtype):
    """Each tile's scores far above the ones before, and the reverse: the running maximum moves by hundreds."""
    c = build(2, [4, 4], [900, 900], 4, 2, 64, 16, dtype, 21, exps=False)
    for row, order in ((0, 1), (1, -1)):
        for p in range(-(-900 // 16)):
            level = p if order > 0 else 56 - p
            c["kc"][c["table"][row][p], :, :, 32:] = q4_ref.e4m3_code(torch.tensor(float(2 ** (level // 8)), dtype=torch.float64))
    check(c, 0.5)
    check(c, -0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_and_small_queries(dtype):
    c = build(1, [6], [400], 4, 2, 64, 32, dtype, 22)
    c["q"][0] *= 1e30
    c["q"][1] *= 1e-30
    c["q"][2] = 0
    c["q"][3, :, 5] = 300.0
    out, lse, status = call(c, 1e-30)
    assert status == 0 and torch.isfinite(out).all() and torch.isfinite(lse).all()
    c["q"][0] *= 1e-30
    check(c, 0.125)


def test_a_nan_query_or_cache_row_shows():
    c = build(2, [2, 1], [200, 200], 4, 2, 64, 32, torch.bfloat16, 23)
    c["q"][0, 1, 3] = math.nan
    c["vc"][c["table"][1][0], 1, 7, 32:] = 0x7F
    out, _, status = call(c, 0.125)
    assert status == 0
    assert out[0, 1].isnan().all() and not out[0, 0].isnan().any() and not out[1].isnan().any()
    assert out[2, 2:].isnan().all() and not out[2, :2].isnan().any()


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 3, 200])
def test_nan_out_of_sight_stays_out(nq, nkv, dh, dtype, window):
    """K and V that are NaN at positions after some of a block's queries, and before the window of others."""
    kv, n = 389, 7
    c = build(2, [n, 2], [kv, 300], nq, nkv, dh, 64, dtype, 29)
    clean, _ = check(c, 0.1, window)

    def poison(pos, which, head, block):
        c[which][c["table"][0][pos // 64], head, pos % 64, dh // 2 + block] = 0x7F if pos % 2 else 0xFF
    poison(kv - 3, "vc", 0, 1)               # the fifth query on sees it
    poison(kv - 1, "kc", 0, 0)               # only the last one does
    if window == 3:
        poison(kv - n - 1, "vc", nkv - 1, 2)  # only the first and the second one do
    out, _, status = call(c, 0.1, window)
    assert status == 0
    G = nq // nkv
    for i in range(n):
        bad = torch.zeros(nq, dh, dtype=torch.bool)
        if i >= 4:
            bad[:G, 16:32] = True
        if i == 6:
            bad[:G] = True
        if window == 3 and i <= 1:
            bad[nq - G:, 32:48] = True
        assert torch.equal(out[i].isnan(), bad), i
        assert torch.equal(out[i][~bad], clean[i][~bad])
    assert torch.equal(out[n:], clean[n:])
    if window == 0:
        poison(5, "vc", nkv - 1, 3)          # far from any border: every query sees it
        out, _, _ = call(c, 0.1, window)
        assert out[:n, nq - G:, 48:64].isnan().all() and not out[:4, nq - G:, :16].isnan().any()


def test_strided_queries_and_a_small_hint():
    c = build(2, [5, 40], [300, 90], 8, 2, 128, 16, torch.bfloat16, 24)
    x = torch.zeros(45, 12, 136, dtype=torch.bfloat16, device="cuda")
    view = x[:, 1:9, 3:131]
    view.copy_(c["q"])
    one, _ = check(c, 0.09, q_dev=view)
    two, _ = check(c, 0.09)
    assert torch.equal(one, two)
    check(c, 0.09, max_q=1)     # rows have more queries than the caller knew
    check(c, 0.09, max_q=1000)


def test_entries_that_are_no_pages_are_not_read():
    c = build(2, [1, 1], [100, 100], 4, 2, 64, 32, torch.bfloat16, 25)
    c["table"][0][1], c["table"][0][2] = -3, 10 ** 6
    out, _, status = call(c, 0.1)
    assert status == 1 << 9 and torch.isfinite(out[0].float()).all()
    d = build(2, [1, 1], [100, 100], 4, 2, 64, 32, torch.bfloat16, 25)
    ref, *_ = call(d, 0.1)
    assert torch.equal(out[1], ref[1])


def test_lengths_and_starts_out_of_range_stay_inside():
    c = build(2, [2, 2], [96, 96], 4, 2, 64, 32, torch.bfloat16, 26)  # whole pages: every slot holds numbers
    c["length"] = [-5, 10 ** 9]
    c["table"] = [[x if x >= 0 else 0 for x in row] for row in c["table"]]
    out, _, status = call(c, 0.1)
    assert status == 1 << 9 and torch.isfinite(out.float()).all() and (out[:2] == 0).all()


def test_without_lse_on_a_stream_and_in_a_graph():
    c = build(3, [2, 2, 2], [1500, 33, 700], 8, 2, 128, 64, torch.bfloat16, 27)
    want, _, _ = call(c, 0.1, want_lse=False)
    side = torch.cuda.Stream()
    got, _, _ = call(c, 0.1, stream=side)
    assert torch.equal(got, want)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache = m.kv_q4_cache(c["kc"].cuda(), c["vc"].cuda(), c["k_exp"].cuda(), c["v_exp"].cuda())
    q, table, start, length = c["q"].cuda(), d(c["table"]), d(c["start"]), d(c["length"])
    out = torch.zeros_like(q)
    ws = torch.empty(m.kv_q4_attend_workspace_bytes(cache, 8, 2, q.dtype), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_q4_attend(cache, q, table, start, length, out, ws, 2, scale=0.1)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_offsets_past_32_bits():
    """Pages behind the 4 GiB mark of caches of 5.4 GB an array."""
    n_pages, nkv, page, dh, L = 9216, 4, 1024, 256, 2100
    small = build(1, [3], [L], 8, nkv, dh, page, torch.bfloat16, 28, exps=False)
    big = []
    for c in (small["kc"], small["vc"]):
        x = torch.zeros((n_pages, nkv, page, 144), dtype=torch.uint8, device="cuda")
        for p, at in zip(small["table"][0][:3], (9215, 3, 8000)):
            x[at] = c[p].cuda()
        big.append(x)
    cache = m.kv_q4_cache(*big)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = small["q"].cuda()
    out = torch.zeros_like(q)
    ws = torch.empty(m.kv_q4_attend_workspace_bytes(cache, 8, 3, q.dtype), dtype=torch.uint8, device="cuda")
    m.kv_q4_attend(cache, q, d([[9215, 3, 8000, -1]]), d([0, 3]), d([L]), out, ws, 3, scale=0.06)
    want, _, _ = call(small, 0.06)
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("nq,nkv,dh,page", [(24, 4, 256, 64), (6, 1, 256, 128), (8, 2, 128, 64), (4, 2, 64, 16)])
@pytest.mark.parametrize("hint", [1, 2, 4, 8, 20])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_repeated_call_gives_the_same_bits(nq, nkv, dh, page, hint, dtype):
    """The cache's rows come from HBM the first time and from L2 after that, when
    copies run at the heels of what they replace: the same work in the same
    order, so the same bits, and the first call's are the plain form's."""
    lens = [7000, 9001, 3333, 12000]
    c = build(4, [4, 3, 4, 1], lens, nq, nkv, dh, page, dtype, dh + hint)
    check(c, 1 / math.sqrt(dh), max_q=hint)
    d = lambda x: (x if torch.is_tensor(x) else torch.tensor(x, dtype=torch.int32)).cuda()
    cache = m.kv_q4_cache(d(c["kc"]), d(c["vc"]), d(c["k_exp"]), d(c["v_exp"]))
    q, table, start, length = d(c["q"]), d(c["table"]), d(c["start"]), d(c["length"])
    ws = torch.empty(m.kv_q4_attend_workspace_bytes(cache, nq, hint, dtype), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(12):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        m.kv_q4_attend(cache, q, table, start, length, out, ws, hint, scale=1 / math.sqrt(dh), lse=lse, status=status)
        outs.append((out, lse))
    assert int(status) == 0
    first = call(c, 1 / math.sqrt(dh), max_q=hint)
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(lse.cpu(), first[1]) and torch.equal(out.cpu(), first[0]), i


@pytest.mark.parametrize("dtype,times", [(torch.float32, 1), (torch.float32, 16), (torch.bfloat16, 16)])
@pytest.mark.parametrize("nq,nkv,dh", HEADS)
def test_long_sums_stay_accurate(nq, nkv, dh, dtype, times):
    """A block sums thousands of positions of positive values by itself (152 rows), the same pages over and over, so
    that the result is that of one turn. The bound on an element: as `check`'s, with a sum over the tiles
    of a share that loses at most 8 steps of 2^-23 a tile for 8 (fp32) or 128 (bf16) tiles and half a step of
    2^-24 for every 8 or 128 tiles after that."""
    page, n_pages, rows = 128, 24, 152
    g = torch.Generator().manual_seed(dh)
    kc, vc = (q4_ref.quantize(x)[0].reshape(n_pages, nkv, page, -1) for x in (
        torch.randn((n_pages * nkv, page, dh), generator=g), torch.randn((n_pages * nkv, page, dh), generator=g).abs()))
    q = torch.randn((3, nq, dh), generator=g).to(dtype)
    c = dict(kc=kc, vc=vc, table=[list(range(n_pages))] * 3, start=[0, 1, 2, 3], length=[n_pages * page] * 3, q=q, k_exp=None, v_exp=None)
    scale = 1 / math.sqrt(dh)
    ref, rlse, spread, reach, _ = q4_ref.attend(q.double(), kc, vc, c["table"], c["start"], c["length"], scale, 0, None, None)
    c.update(table=[list(range(n_pages)) * times] * rows, start=list(range(rows + 1)), length=[n_pages * page * times] * rows,
             q=q.repeat(51, 1, 1)[:rows])
    out, lse, status = call(c, scale)
    assert status == 0
    wide = dtype == torch.float32
    far, tiles = (8, n_pages * times) if wide else (128, n_pages * times)
    lost = 8 * min(far, tiles) * 2.0 ** -23 + tiles / far * 2.0 ** -24
    d = ((2.0 ** -21 if wide else 2.0 ** -16) + dh * 2.0 ** -24) * reach
    rel = 2 * d + 2.0 ** -21 + (2.0 ** -22 if wide else 2.0 ** -11)
    tol = ref.abs() * (2.0 ** -24 if wide else 2.0 ** -8) + (rel[..., None] + lost) * spread * (1 + 2.0 ** -8)
    ltol = d + 2.0 ** -20 + (rlse.abs() + math.log(times)) * 2.0 ** -23 + tiles * 2.0 ** -24
    for r in range(rows):
        assert ((out[r].double() - ref[r % 3]).abs() <= tol[r % 3]).all(), r
        assert ((lse[r].double() - rlse[r % 3] - math.log(times)).abs() <= ltol[r % 3]).all(), r
