"""kv_attend_prompt against plain 64-bit attention.

Bounds (derived, then fixed): a score is a sum of dh exact products (bf16) or of
rounded ones (fp32) in fp32, off by at most d = dh 2^-23 scale sum |q k| in any
order (2^-23: the tensor core drops the bits past fp32's), and by 2^-24 of
itself by its factor. A weight is off by 2 d + 2^-21 of itself and, for bf16, by
its rounding to bf16, 2^-8; the sum of the weights and that of the products with v over n
positions by n 2^-23 of their sizes; an output by its type's half step; lse by
d + 2^-20 + n 2^-24 and 2^-23 of itself."""
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import tree_ref

pytestmark = pytest.mark.gpu


def make(n, nq, nkv, dh, dtype, seed, q_scale=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((sum(n), nq + 2 * nkv, dh), generator=g)
    x[:, :nq] *= q_scale
    x = x.to(dtype)
    return dict(x=x, nq=nq, nkv=nkv, start=[sum(n[:r]) for r in range(len(n) + 1)])


def parts(c, x=None):
    x = c["x"] if x is None else x
    return x[:, :c["nq"]], x[:, c["nq"]:c["nq"] + c["nkv"]], x[:, c["nq"] + c["nkv"]:]


def call(c, scale, window=0, max_len=None, want_lse=True, stream=None, qkv=None, start=None):
    q, k, v = qkv or parts(c, c["x"].cuda())
    T, nq, dh = q.shape
    start = c["start"] if start is None else start
    out = torch.full((T, nq, dh), 77.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, nq), 77.0, device="cuda") if want_lse else None
    ws = torch.full((m.kv_attend_prompt_workspace_bytes(T, len(start) - 1),), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_len = max_len or max(1, max(b - a for a, b in zip(start, start[1:])))
    m.kv_attend_prompt(q, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), out, ws, max_len, scale=scale, window=window, lse=lse,
                       status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu(), int(status)


def check(c, scale, window=0, **kw):
    out, lse, status = call(c, scale, window, **kw)
    assert status == 0
    q, k, v = parts(c)
    ref, rlse, spread, reach = tree_ref.prompt(q.double(), k.double(), v.double(), c["start"], scale, window)
    wide, dh = q.dtype == torch.float32, q.shape[2]
    n = max([b - a for a, b in zip(c["start"], c["start"][1:])] + [1])
    n = min(n, window) if window else n
    d = (dh * 2.0 ** -23 + 2.0 ** -24) * reach
    rel = 2 * d + 2.0 ** -21 + n * 2.0 ** -22 + (0 if wide else 2.0 ** -8)
    tol = ref.abs() * (2.0 ** -24 if wide else 2.0 ** -8) + rel[..., None] * spread * (1 + 2.0 ** -7) + 1e-37
    a, b = c["start"][0], c["start"][-1]
    off = (out.double() - ref).abs()
    assert (off <= tol)[a:b].all(), (float((off / tol)[a:b].max()), (off > tol).nonzero()[:5])
    assert ((lse.double() - rlse).abs() <= d + 2.0 ** -20 + n * 2.0 ** -24 + rlse.abs() * 2.0 ** -23)[a:b].all()
    assert (out[:a] == 77).all() and (out[b:] == 77).all() and (lse[:a] == 77).all() and (lse[b:] == 77).all()
    return out, lse


HEADS = [(4, 2, 64), (8, 2, 128), (24, 4, 256), (5, 5, 64), (3, 3, 256), (16, 1, 128)]


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_rows_of_all_lengths(nq, nkv, dh, dtype):
    """Lengths of zero and one, around tiles of 32, 64, 128 and 256, packed side by side."""
    check(make([1, 0, 2, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 5, 255, 256, 257, 0], nq, nkv, dh, dtype, dh), 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS[:3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_rows(nq, nkv, dh, dtype):
    check(make([1500, 3, 777], nq, nkv, dh, dtype, dh + 1), 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS[:3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 127, 128, 129, 300, 5000, 2 ** 31 - 1])
def test_windows(nq, nkv, dh, dtype, window):
    check(make([600, 5, 129, 333], nq, nkv, dh, dtype, window % 1000), 1 / math.sqrt(dh), window)


@pytest.mark.parametrize("n,nq,nkv,dh", [([131, 1, 70], 4, 2, 64), ([17, 90], 8, 2, 128), ([64, 300], 3, 3, 256),
                                         ([700], 4, 2, 64), ([33, 367], 8, 2, 128), ([900], 3, 1, 256)])
@pytest.mark.parametrize("window", [0, 50])
def test_few_queries_take_small_tiles(n, nq, nkv, dh, window):
    """fp32: tiles of 16 queries where those are no more than the SMs, of 32 where those are few."""
    check(make(n, nq, nkv, dh, torch.float32, dh + len(n)), 1 / math.sqrt(dh), window)


def test_one_token():
    for dtype in (torch.bfloat16, torch.float32):
        c = make([1], 4, 2, 64, dtype, 3)
        out, _ = check(c, 0.1)
        assert torch.equal(out, parts(c)[2].repeat_interleave(2, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [100, 4096])
def test_many_rows(rows, dtype):
    n = [(r * 7919) % 41 if rows == 100 else (r * 7919) % 4 for r in range(rows)]
    check(make(n, 4, 2, 64, dtype, rows), 0.125)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scores_that_rise_and_fall(dtype):
    """The running maximum moves by hundreds along the keys, or never after the first."""
    for sign in (1, -1):
        c = make([700], 4, 2, 64, dtype, 21)
        q, k, v = parts(c)
        k[:, :, 0] = (torch.arange(700) * sign).to(dtype)[:, None]
        q[:, :, 0] = 4
        check(c, 0.25)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_and_small_scores(dtype):
    c = make([300], 4, 2, 64, dtype, 22)
    check(c, 0.0)
    check(c, -0.2)
    c["x"][:, :4] *= 1e-30
    check(c, 0.125)
    c = make([300], 4, 2, 64, dtype, 22)
    c["x"][:, :6] *= 1e15
    out, lse, status = call(c, 1e-28)
    assert status == 0 and torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("nq,nkv,dh", HEADS[:3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 70])
def test_what_is_out_of_sight_may_be_anything(nq, nkv, dh, dtype, bad, window):
    """NaN and infinities in K and V reach the queries that see them and no others: not earlier ones, not other rows,
    not those whose window has passed."""
    n = [200, 150, 70]
    c = make(n, nq, nkv, dh, dtype, 29)
    clean, _ = check(c, 0.1, window)
    _, k, v = parts(c)
    v[100, 0, 5] = bad              # row 0, position 100
    v[200, nkv - 1, 3] = bad        # row 1's first position
    k[349, 0, 2] = math.nan         # row 1's last one
    v[199, nkv - 1, dh - 1] = bad   # row 0's last one
    out, _, status = call(c, 0.1, window)
    assert status == 0
    G = nq // nkv
    want = torch.zeros_like(out, dtype=torch.bool)
    w = window or 1 << 30
    want[100:min(200, 100 + w), :G, 5] = True
    want[200:min(350, 200 + w), nq - G:, 3] = True
    want[349, :G] = True
    want[199, nq - G:, dh - 1] = True
    assert torch.equal(~torch.isfinite(out), want), (~torch.isfinite(out) ^ want).nonzero()[:5]
    assert torch.equal(out[~want], clean[~want])


def test_infinite_keys():
    """A score of -inf weighs nothing; a row with nothing else gives zeros; +inf and NaN make NaN."""
    c = make([4], 1, 1, 64, torch.bfloat16, 30)
    q, k, v = parts(c)
    q[:, :, 0] = 1.0
    k[0, 0, 0] = -math.inf
    out, lse, _ = call(c, 1.0)
    assert (out[0] == 0).all() and lse[0] == -math.inf and torch.isfinite(out[1:]).all() and torch.isfinite(lse[1:]).all()
    assert torch.equal(out[1, 0], v[1, 0])
    k[0, 0, 0] = math.inf
    assert call(c, 1.0)[0].isnan().all()


def test_separate_and_padded_tensors_streams_and_graphs():
    c = make([90, 300], 8, 2, 128, torch.bfloat16, 31)
    want, wl = check(c, 0.09)
    q, k, v = (t.contiguous().cuda() for t in parts(c))
    assert torch.equal(call(c, 0.09, qkv=(q, k, v))[0], want)
    wide = torch.zeros(390, 9, 136, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 1:9, 8:136]
    view.copy_(q)
    heads_first = k.transpose(0, 1).contiguous().transpose(0, 1)
    got, gl, _ = call(c, 0.09, qkv=(view, heads_first, v), stream=torch.cuda.Stream(), max_len=1)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    start = torch.tensor(c["start"], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(m.kv_attend_prompt_workspace_bytes(390, 2), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_attend_prompt(q, k, v, start, out, ws, 300, scale=0.09)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("nq,nkv,dh", [(256, 1, 64), (125, 1, 128), (129, 1, 64), (1021, 1, 64), (1024, 8, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_heads_to_a_kv_head(nq, nkv, dh, dtype):
    """More than a query tile holds (parts of them that divide their number), one head at a time where that is prime."""
    check(make([3, 0, 34], nq, nkv, dh, dtype, nq), 1 / math.sqrt(dh))


@pytest.mark.parametrize("nq,nkv,dh", HEADS[:3])
def test_two_calls_at_once(nq, nkv, dh):
    """On two streams, one workspace between them."""
    cs = [make([900, 5, 300], nq, nkv, dh, torch.bfloat16, 41), make([31, 700], nq, nkv, dh, torch.bfloat16, 42)]
    want = [check(c, 0.08)[0] for c in cs]
    ws = torch.empty(m.kv_attend_prompt_workspace_bytes(2000, 3), dtype=torch.uint8, device="cuda")
    args = []
    for c in cs:
        q, k, v = parts(c, c["x"].cuda())
        args.append((q, k, v, torch.tensor(c["start"], dtype=torch.int32, device="cuda"), torch.zeros(q.shape, dtype=q.dtype, device="cuda"), ws, 900))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s in zip(args, streams):
            m.kv_attend_prompt(*a, scale=0.08, stream=s)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert torch.equal(a[4].cpu(), w)


def test_padded_batches_and_starts_out_of_range():
    """Positions before the first row and behind the last are left alone; starts out of range stay inside."""
    c = make([40, 50, 60, 30], 4, 2, 64, torch.bfloat16, 32)
    full, _ = check(c, 0.1)
    c["start"] = c["start"][1:4]
    part, _ = check(c, 0.1)
    assert torch.equal(part[40:150], full[40:150])
    out, _, status = call(c, 0.1, start=[-100, 40, 10 ** 9])
    assert status == 0 and torch.isfinite(out.float()).all() and torch.equal(out[:40], full[:40])
    out, _, _ = call(c, 0.1, start=[90, 40, 60])  # descending: an empty row
    assert (out[:40] == 77).all()


@pytest.mark.parametrize("nq,nkv,dh", HEADS[:3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_repeated_call_gives_the_same_bits(nq, nkv, dh, dtype):
    c = make([1000, 17, 600, 255], nq, nkv, dh, dtype, 33)
    first = check(c, 1 / math.sqrt(dh))
    x = c["x"].cuda()
    q, k, v = parts(c, x)
    start = torch.tensor(c["start"], dtype=torch.int32, device="cuda")
    ws = torch.empty(m.kv_attend_prompt_workspace_bytes(q.shape[0], 4), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(12):
        out, lse = torch.empty(q.shape, dtype=dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        m.kv_attend_prompt(q, k, v, start, out, ws, 1000, scale=1 / math.sqrt(dh), lse=lse)
        outs.append((out, lse))
    for i, (out, lse) in enumerate(outs):
        assert torch.equal(out.cpu(), first[0]) and torch.equal(lse.cpu(), first[1]), i


def test_offsets_past_32_bits():
    """Rows that lie 2^31 elements apart."""
    c = make([3], 4, 2, 64, torch.bfloat16, 34)
    want, _ = check(c, 0.1)
    flat = torch.zeros(2 * (1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((3, 8, 64), (1 << 31, 64, 1))
    x.copy_(c["x"].cuda())
    assert torch.equal(call(c, 0.1, qkv=parts(c, x))[0], want)
