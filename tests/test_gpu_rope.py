"""kv_q4_append_rope against plain 64-bit norms and rotations, and against
kv_q4_append for what the cache holds.

Bounds (derived, then fixed): the sum of dh squares is fp32 in any order, off by
at most 16 roundings of 2^-24 (8 elements a lane or 8 strided ones, then five
exchanges, the mean and eps); half of that reaches its root, whose own error is
2 steps (2^-22); with the two products y is off by 2^-20 of itself. cos and sin
are off by 2 steps of 2^-24, by the 24 bits of their argument (2^-24 pi / 4) and by
the frequency's 2^-53, 2 pi pos 2^-55 of a turn: 2^-22 up to position 2^30. A
rotated element is a c - b s in two roundings: off by (|a| + |b|) 2^-19, and by
its type's half step. What the cache keeps of a key is rounded from a value that
is off by (|a| + |b|) 2^-28 at most (two floats: products and sums of some ten terms in
2^-32 each), so its bytes are those of the 64-bit value, or of that moved by
2^-28 either way where a border lies between."""
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref, tree_ref

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
NONFINITE, BAD = 1 << 10, 1 << 9


def make(tokens, nq, nkv, dh, dtype, seed, page=16, far=30000, norm=True, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((tokens, nq + 2 * nkv, dh), generator=g) * torch.exp(torch.randn((1, nq + 2 * nkv, dh), generator=g))).to(dtype)
    n_pages = -(-tokens // page) + 1
    w = lambda: 1 + 0.1 * torch.randn(dh, generator=g) if norm else None
    c = dict(q=x[:, :nq], k=x[:, nq:nq + nkv], v=x[:, nq + nkv:], slot=torch.randperm(n_pages * page, generator=g)[:tokens].int(),
             pos=torch.randint(0, far, (tokens,), generator=g).int(), q_norm=w(), k_norm=w(), page=page, n_pages=n_pages,
             k_exp=torch.tensor([h % 4 - 3 for h in range(nkv)], dtype=torch.int32), v_exp=torch.tensor([h % 5 - 1 for h in range(nkv)], dtype=torch.int32))
    if not fused:
        c.update({n: c[n].contiguous() for n in "qkv"})
    return c


def dev(c):
    fused = c["q"]._base is not None and c["k"]._base is c["q"]._base
    out = {n: t.cuda() if torch.is_tensor(t) else t for n, t in c.items()}
    if fused:  # the slices of one projection, on the device too
        x, nq, nkv = c["q"]._base.cuda(), c["q"].shape[1], c["k"].shape[1]
        out.update(q=x[:, :nq], k=x[:, nq:nq + nkv], v=x[:, nq + nkv:])
    return out


def call(c, rope, eps=1e-6, with_k=True, **kw):
    d = dev(c)
    T, nkv, dh = d["k"].shape
    shape = (c["n_pages"], nkv, c["page"], dh * 9 // 16)
    kc, vc = (torch.full(shape, 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = m.kv_q4_cache(kc, vc, d["k_exp"], d["v_exp"])
    q_out = torch.full(d["q"].shape, 77.0, dtype=d["q"].dtype, device="cuda")
    k_out = torch.full(d["k"].shape, 77.0, dtype=d["q"].dtype, device="cuda") if with_k else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_append_rope(cache, d["q"], d["k"], d["v"], rope, d["pos"], d["slot"], q_out, k_out=k_out, q_norm=d["q_norm"], k_norm=d["k_norm"],
                        eps=eps, status=status, **kw)
    torch.cuda.synchronize()
    return q_out.cpu(), None if k_out is None else k_out.cpu(), kc.cpu(), vc.cpu(), int(status)


def rows_of(cache, slot, page):
    s = slot.long()
    return cache[s // page, :, s % page]


def quantize64(x, exp):
    """Bytes of 64-bit values, the scales' quotients in 64 bits too."""
    y = (x * (2.0 ** -exp.double())[:, None]).unflatten(-1, (-1, 16))
    scale = q4_ref.e4m3_round(y.abs().amax(-1, keepdim=True) / 6)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: argmin keeps the first of equals
    code = order[(y.abs().unsqueeze(-1) - q4_ref.LEVELS * scale.unsqueeze(-1)).abs()[..., order].argmin(-1)]
    nib = torch.where(scale > 0, code + 8 * torch.signbit(y), 0).to(torch.uint8).flatten(-2)
    return torch.cat([nib[..., 0::2] | (nib[..., 1::2] << 4), q4_ref.e4m3_code(scale.squeeze(-1))], -1)


def freqs(rot, theta):
    return theta ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))


def check(c, rot, theta=1e4, eps=1e-6, freq=None):
    dtype = c["q"].dtype
    rope = m.mtp_rope(rot, theta) if freq is None else m.mtp_rope(rot, freq=freq.tolist())
    f = freqs(rot, theta) if freq is None else freq
    q, k, kc, vc, status = call(c, rope, eps)
    assert status == 0
    for got, x, w in ((q, c["q"], c["q_norm"]), (k, c["k"], c["k_norm"])):
        y, z = tree_ref.turned(x.double(), w, c["pos"], rot, f, eps)
        size = y.abs().clone()
        size[..., :rot // 2] += y[..., rot // 2:rot].abs()
        size[..., rot // 2:rot] += y[..., :rot // 2].abs()
        tol = size * 2.0 ** -19 + z.abs() * HALF[dtype] * (1 + 2.0 ** -8) + 1e-37
        off = (got.double() - z).abs()
        assert (off <= tol).all(), (float((off / tol).max()), (off > tol).nonzero()[:5])
    # the cache: V as kv_q4_append has it, K by its values' bounds (y, z and size are its own)
    raw, _ = q4_ref.quantize(c["v"].float(), c["v_exp"])
    assert torch.equal(rows_of(vc, c["slot"], c["page"]), raw)
    dh, got = y.shape[-1], rows_of(kc, c["slot"], c["page"])
    near = [quantize64(z + size * by * 2.0 ** -28, c["k_exp"]) for by in (0, -1, 1)]
    split = lambda raw: (torch.stack([raw[..., :dh // 2] & 15, raw[..., :dh // 2] >> 4], -1).flatten(-2).unflatten(-1, (-1, 16)), raw[..., dh // 2:, None])
    code, scale = split(got)
    fits = torch.zeros(code.shape[:-1], dtype=torch.bool)
    for raw in near:
        fits |= ((split(raw)[0] == code).all(-1) & (split(raw)[1] == scale).squeeze(-1))
    assert fits.all(), (~fits).nonzero()[:5]
    assert (near[0] != got).float().mean() < 1e-3
    used = torch.zeros(kc.shape[0] * c["page"], dtype=torch.bool)
    used[c["slot"].long()] = True
    assert (kc.transpose(1, 2).flatten(0, 1)[~used] == 0xEE).all()  # other slots are left alone
    return q, k


HEADS = [(4, 2, 64), (8, 2, 128), (24, 4, 256), (5, 5, 64), (1, 1, 128)]


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
def test_whole_and_partial_rotations(nq, nkv, dh, dtype, norm):
    for rot in (0, 2, 16, 32, 34, dh // 2, dh - 2, dh):
        check(make(11, nq, nkv, dh, dtype, dh + rot, norm=norm), rot)


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 33, 257])
@pytest.mark.parametrize("nq,nkv,dh", HEADS)
def test_counts_around_a_block(tokens, nq, nkv, dh):
    check(make(tokens, nq, nkv, dh, torch.bfloat16, tokens), dh)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("theta", [1e4, 1e7])
def test_far_positions(dtype, theta):
    c = make(64, 4, 2, 128, dtype, 5, far=1 << 30)
    c["pos"][:4] = torch.tensor([0, 1, (1 << 30) - 1, 1 << 29])
    check(c, 128, theta)
    check(c, 126, theta)


def test_scaled_frequencies_and_contiguous_rows():
    f = torch.tensor([0.37, 1.9, 0.0, 2 * math.pi, 0.001, 3.0, -0.5, 1e-6] * 2, dtype=torch.float64)
    check(make(9, 4, 2, 64, torch.float32, 6, fused=False, far=5000), 32, freq=f)


@pytest.mark.parametrize("dh,rot", [(64, 64), (128, 32), (256, 254), (256, 0)])
def test_odd_strides_and_alignment(dh, rot):
    """The rows of the general kernel: strides that no vector load takes."""
    c = make(13, 3, 3, dh, torch.bfloat16, 7)
    want = call(c, m.mtp_rope(rot))
    x = torch.zeros(13, 11, dh + 3, dtype=torch.bfloat16, device="cuda")
    d = dev(c)
    views = [x[:, a:a + 3, 1:dh + 1] for a in (1, 4, 7)]
    for v, n in zip(views, "qkv"):
        v.copy_(d[n])
    kc, vc = (torch.full(want[2].shape, 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2))
    q, k = torch.empty(13, 3, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(13, 3, dh, dtype=torch.bfloat16, device="cuda")
    m.kv_q4_append_rope(m.kv_q4_cache(kc, vc, d["k_exp"], d["v_exp"]), *views, m.mtp_rope(rot), d["pos"], d["slot"], q, k_out=k,
                        q_norm=d["q_norm"], k_norm=d["k_norm"])
    y, z = tree_ref.turned(c["q"].double(), c["q_norm"], c["pos"], rot, freqs(rot, 1e4), 1e-6)
    assert (q.cpu().double() - z).abs().max() <= 2.0 ** -7 * z.abs().max()
    # the two kernels' sums go in another order: a code may sit on another side of its border, no more
    other = (rows_of(kc.cpu(), c["slot"], 16) != rows_of(want[2], c["slot"], 16)).float().mean()
    assert other < 1e-3 and torch.equal(vc.cpu(), want[3])


@pytest.mark.parametrize("dh,rot", [(64, 32), (256, 256), (128, 18)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding_and_refused_rows(dh, rot, dtype):
    c = make(40, 4, 2, dh, dtype, 8)
    good = call(c, m.mtp_rope(rot))
    c["pos"] = c["pos"].clone()
    keep = c["slot"].clone()
    c["slot"] = c["slot"].clone()
    c["slot"][3] = -1                                  # refused by the plan: rotated, not appended
    c["pos"][5] = c["slot"][5] = -1                    # padding
    c["pos"][39] = c["slot"][39] = -1
    q, k, kc, vc, status = call(c, m.mtp_rope(rot))
    assert status == 0
    assert torch.equal(q[3], good[0][3]) and torch.equal(k[3], good[1][3])
    assert (q[[5, 39]] == 0).all() and (k[[5, 39]] == 0).all()
    live = torch.ones(40, dtype=torch.bool)
    live[[3, 5, 39]] = False
    assert torch.equal(q[live], good[0][live]) and torch.equal(rows_of(kc, keep, 16)[live], rows_of(good[2], keep, 16)[live])
    assert (rows_of(kc, keep, 16)[~live] == 0xEE).all() and (rows_of(vc, keep, 16)[~live] == 0xEE).all()
    for t, s in ((7, c["n_pages"] * 16), (9, -2)):
        bad = {**c, "slot": c["slot"].clone()}
        bad["slot"][t] = s
        assert call(bad, m.mtp_rope(rot))[4] == BAD
    bad = {**c, "pos": c["pos"].clone()}
    bad["pos"][11] = -7                                # a slot beside a position below 0
    q, _, kc, _, status = call(bad, m.mtp_rope(rot))
    assert status == BAD and (q[11] == 0).all() and (rows_of(kc, keep, 16)[11] == 0xEE).all()


@pytest.mark.parametrize("rot", [128, 6])
@pytest.mark.parametrize("norm", [True, False])
def test_what_is_not_finite_shows(rot, norm):
    c = make(6, 4, 2, 128, torch.float32, 9, norm=norm)
    x = c["q"]._base
    clean = call(c, m.mtp_rope(rot))
    x[1, 4, 70] = math.nan    # a key
    x[2, 7, 17] = math.inf    # a value
    x[3, 1, 3] = math.nan     # a query
    q, k, kc, vc, status = call(c, m.mtp_rope(rot))
    assert status == NONFINITE
    krow, vrow = rows_of(kc, c["slot"], 16), rows_of(vc, c["slot"], 16)
    hit = torch.tensor([True] * 8 if norm else [b in ((0, 4) if rot == 128 else (4,)) for b in range(8)])
    assert torch.equal(krow[1, 0, 64:] == 0x7F, hit) and (krow[1, 0, 64:72][hit] == 0x7F).all()
    assert vrow[2, 1, 64:].tolist().count(0x7F) == 1 and vrow[2, 1, 65] == 0x7F
    assert q[3, 1].isnan().any() and torch.equal(q[3, [0, 2, 3]], clean[0][3, [0, 2, 3]])
    rest = [0, 4, 5]
    assert torch.equal(q[rest], clean[0][rest]) and torch.equal(krow[rest], rows_of(clean[2], c["slot"], 16)[rest])


def test_values_past_the_range_by_the_exponent_saturate():
    c = make(3, 2, 1, 64, torch.float32, 10, norm=False)
    c["q"]._base[:, 2:] *= 1e30
    c["k_exp"][:] = -64
    c["v_exp"][:] = -64
    _, _, kc, vc, status = call(c, m.mtp_rope(64))
    assert status == 0
    cache = [torch.full(kc.shape, 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2)]
    d = dev(c)
    m.kv_q4_append(m.kv_q4_cache(*cache, d["k_exp"], d["v_exp"]), d["k"], d["v"], d["slot"])
    assert torch.equal(cache[1].cpu(), vc)


@pytest.mark.parametrize("dh,rot", [(128, 128), (64, 20)])
def test_in_place_on_a_stream_and_in_a_graph(dh, rot):
    c = make(70, 4, 2, dh, torch.bfloat16, 11, fused=False)
    rope = m.mtp_rope(rot)
    want = call(c, rope)
    side = torch.cuda.Stream()
    got = call(c, rope, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))
    assert torch.equal(call(c, rope, with_k=False)[2], want[2])
    d = dev(c)
    kc, vc = (torch.full(want[2].shape, 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = m.kv_q4_cache(kc, vc, d["k_exp"], d["v_exp"])
    q, k = d["q"].clone(), d["k"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_q4_append_rope(cache, q, k, d["v"], rope, d["pos"], d["slot"], q, k_out=k, q_norm=d["q_norm"], k_norm=d["k_norm"])
    del rope
    for _ in range(2):
        q.copy_(d["q"])
        k.copy_(d["k"])
        kc.fill_(0xEE)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.cpu(), want[0]) and torch.equal(k.cpu(), want[1]) and torch.equal(kc.cpu(), want[2])


def test_offsets_past_32_bits():
    """A slot behind the 4 GiB mark, and rows of a projection that lie 2^31 elements apart."""
    n_pages, nkv, page, dh = 9216, 4, 1024, 256
    c = make(2, 4, nkv, dh, torch.bfloat16, 12, fused=False)
    c.update(page=page)
    small = call({**c, "slot": torch.tensor([3, 17], dtype=torch.int32), "n_pages": 1}, m.mtp_rope(dh))
    kc, vc = (torch.zeros((n_pages, nkv, page, 144), dtype=torch.uint8, device="cuda") for _ in range(2))
    d = dev(c)
    wide = torch.zeros(((1 << 31) + 8192,), dtype=torch.bfloat16, device="cuda")
    q = wide.as_strided((2, 4, dh), (1 << 31, dh, 1))
    q.copy_(d["q"])
    slot = torch.tensor([9215 * page + 3, 5 * page + 17], dtype=torch.int32, device="cuda")
    out = torch.empty_like(d["q"])
    m.kv_q4_append_rope(m.kv_q4_cache(kc, vc, d["k_exp"], d["v_exp"]), q, d["k"], d["v"], m.mtp_rope(dh), d["pos"], slot, out,
                        q_norm=d["q_norm"], k_norm=d["k_norm"])
    assert torch.equal(out.cpu(), small[0])
    assert torch.equal(kc[9215, :, 3].cpu(), small[2][0, :, 3]) and torch.equal(vc[5, :, 17].cpu(), small[3][0, :, 17])
