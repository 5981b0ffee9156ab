"""Refusals of the paged 4-bit cache's entry points and of spec_logprobs that
need no GPU (nothing is launched), and the plain implementations that the GPU
tests compare with, pinned against PyTorch and worked examples."""
import ctypes
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref

FAKE = 0x10000  # never dereferenced
BAD = 9


@pytest.fixture(scope="module")
def L():
    from mtp_speculative_decoding_step_gb300 import _build
    _build.build()
    return m.lib()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_exp=None, v_exp=None, n_kv=2, head_dim=128, page=16, n_pages=8)
    d.update(kw)
    return ctypes.byref(m.Q4Cache(*[d[n] for n, _ in m.Q4Cache._fields_]))


def test_row_bytes(L):
    assert [m.kv_q4_row_bytes(d) for d in (64, 128, 256)] == [36, 72, 144]
    assert [m.kv_q4_row_bytes(d) for d in (0, 32, 96, 512, -64)] == [0] * 5


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(head_dim=96), dict(n_kv=0),
              dict(page=0), dict(page=8), dict(page=24), dict(n_pages=0), dict(page=1 << 20, n_pages=1 << 11)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(L, kw):
    c = _cache(**kw)
    assert L.kv_q4_append(None, c, 1, FAKE, 256, 128, FAKE, 256, 128, 1, FAKE, None) == BAD
    assert L.kv_q4_read(None, c, 1, FAKE, FAKE, FAKE, 1, None) == BAD
    assert L.kv_q4_attend(None, c, 1, 4, 1, FAKE, 512, 128, 1, FAKE, 4, FAKE, FAKE, 1, 0.1, 0, FAKE, None, None,
                          FAKE) == BAD


@pytest.mark.parametrize("at,val", [(2, -1), (3, None), (6, None), (9, 2), (9, 7), (10, None), (3, FAKE + 1)])
def test_append_refuses(L, at, val):
    args = [None, _cache(), 1, FAKE, 256, 128, FAKE, 256, 128, 1, FAKE, None]
    args[at] = val
    assert L.kv_q4_append(*args) == BAD


@pytest.mark.parametrize("at,val", [(2, -1), (3, None), (4, None), (5, None), (4, FAKE + 4), (6, 3)])
def test_read_refuses(L, at, val):
    args = [None, _cache(), 1, FAKE, FAKE, FAKE, 1, None]
    args[at] = val
    assert L.kv_q4_read(*args) == BAD


def test_nothing_to_do_is_not_an_error(L):
    c = _cache()
    assert L.kv_q4_append(None, c, 0, None, 0, 0, None, 0, 0, 1, None, None) == 0
    assert L.kv_q4_read(None, c, 0, None, None, None, 1, None) == 0
    assert L.kv_q4_attend(None, c, 1, 4, 0, None, 0, 0, 1, None, 4, None, None, 1, 0.1, 0, None, None, None, None) == 0
    assert L.spec_logprobs(None, 0, 100, None, 100, 0, None, 0, None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("at,val", [
    (2, 0), (2, 4097), (3, 0), (3, 5), (4, -1), (5, None), (5, FAKE + 1), (8, 2), (9, None), (10, 0), (10, 1 << 28),
    (11, None), (12, None), (13, 0), (14, math.inf), (14, math.nan), (15, -1), (16, None), (16, FAKE + 8), (19, None),
    (19, FAKE + 4)])
def test_attend_refuses(L, at, val):
    args = [None, _cache(), 1, 4, 1, FAKE, 512, 128, 1, FAKE, 4, FAKE, FAKE, 1, 0.1, 0, FAKE, None, None, FAKE]
    args[at] = val
    assert L.kv_q4_attend(*args) == BAD


def test_workspace_queries(L):
    assert L.kv_q4_attend_workspace_bytes(_cache(), 8, 4, 1) > 0
    assert L.kv_q4_attend_workspace_bytes(_cache(head_dim=80), 8, 4, 1) == 0
    assert L.kv_q4_attend_workspace_bytes(_cache(), 8, 0, 1) == 0
    assert L.kv_q4_attend_workspace_bytes(_cache(), 8, 4, 5) == 0
    assert m.spec_logprobs_workspace_bytes(4, 1000, 5) > 0
    assert [m.spec_logprobs_workspace_bytes(*a) for a in ((0, 10, 1), (1, 0, 1), (1, 10, 65), (1, 10, -1))] == [0] * 4


@pytest.mark.parametrize("at,val", [
    (1, 0), (1, 4097), (2, 0), (2, 24), (3, 0), (4, 0), (5, -1), (6, None), (7, None), (8, None), (9, None),
    (10, None), (11, None), (12, None), (13, None), (14, None), (11, FAKE + 4),  # overlaps cover
    (3, 1 << 30), (4, 1 << 28)])
def test_plan_refuses(L, at, val):
    #       stream rows page maxp pages toks cover  keep new   table free cover_out start slot pos status
    args = [None, 2, 16, 8, 32, 10, FAKE, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, FAKE, FAKE, FAKE, None]
    args[at] = val
    assert L.kv_page_plan(*args) == BAD


@pytest.mark.parametrize("at,val", [(1, -1), (2, 0), (2, (1 << 20) + 1), (3, None), (3, FAKE + 2), (4, 99), (5, 2),
                                    (6, None), (7, -1), (7, 65), (8, None), (11, None), (12, None), (14, None),
                                    (14, FAKE + 8)])
def test_logprobs_refuses(L, at, val):
    args = [None, 2, 100, FAKE, 100, 0, FAKE, 3, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]
    args[at] = val
    assert L.spec_logprobs(*args) == BAD


def test_binding_refuses_wrong_shapes_and_types(L):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(m.MTPError):
        m.kv_q4_cache(u8(4, 2, 16, 70), u8(4, 2, 16, 70))
    with pytest.raises(m.MTPError):
        m.kv_q4_cache(u8(4, 2, 16, 72), u8(4, 2, 16, 72).transpose(0, 1))
    with pytest.raises(m.MTPError):
        m.kv_q4_cache(u8(4, 2, 16, 72), u8(4, 2, 16, 72), k_exp=i32(3))
    c = m.kv_q4_cache(u8(4, 2, 16, 72), u8(4, 2, 16, 72))
    assert (c.c.head_dim, c.c.n_kv, c.c.page, c.c.n_pages) == (128, 2, 16, 4)
    x = torch.zeros(3, 2, 128)
    with pytest.raises(m.MTPError):
        m.kv_q4_append(c, x, x[:, :1], i32(3), stream=0)
    with pytest.raises(m.MTPError):
        m.kv_q4_append(c, x, x.half(), i32(3), stream=0)
    with pytest.raises(m.MTPError):
        m.kv_q4_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x, i32(3), stream=0)
    with pytest.raises(m.MTPError):
        m.kv_q4_read(c, i32(3).long(), x, x, stream=0)
    q, ws = torch.zeros(3, 4, 128), u8(1 << 26)
    ok = dict(max_q=3, scale=1.0, stream=0)
    with pytest.raises(m.MTPError):
        m.kv_q4_attend(c, q, i32(1, 4), i32(3), i32(1), q, ws, **ok)       # start of two rows
    with pytest.raises(m.MTPError):
        m.kv_q4_attend(c, q, i32(1, 4), i32(2), i32(1), q.bfloat16(), ws, **ok)
    with pytest.raises(m.MTPError):
        m.kv_q4_attend(c, q, i32(1, 4), i32(2), i32(1), q, ws[:16], **ok)  # short workspace
    with pytest.raises(m.MTPError):
        m.kv_page_plan(i32(2), i32(2), i32(2), i32(2, 4), i32(8), i32(2), i32(2), i32(4), i32(4), 16, stream=0)
    with pytest.raises(m.MTPError):
        m.spec_logprobs(torch.zeros(2, 100), i32(2), torch.zeros(2), u8(1 << 20), top_id=i32(2, 3), stream=0)


# ------------------------------------------------------------------ the plain implementations

def test_ref_scales_match_pytorch_and_every_code_reads_back():
    x = torch.cat([torch.rand(4000, dtype=torch.float64) * 500, 2.0 ** torch.arange(-12, 9).double()])
    want = x.float().clamp(max=448).to(torch.float8_e4m3fn).float().double()
    assert torch.equal(q4_ref.e4m3_round(x.float().double()), want)
    raw = torch.zeros(1, 36, dtype=torch.uint8)
    raw[0, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE])
    raw[0, 32:] = q4_ref.e4m3_code(torch.tensor([2.0, 1.0, 1.0, 1.0], dtype=torch.float64))
    assert q4_ref.values(raw, 64)[0, :16].tolist() == [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]


def test_ref_rounding_worked_example():
    x = torch.zeros(1, 1, 64, dtype=torch.float64)
    x[0, 0, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])  # scale 1: every border
    x[0, 0, 8:12] = torch.tensor([-0.26, -4.9, 0.2, 5.1])
    raw, val = q4_ref.quantize(x)
    assert val[0, 0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -4, 0, 6]
    assert torch.equal(q4_ref.values(raw, 64), val)


def test_ref_plan_worked_example():
    # three rows on pages of 16: the first gives a page back, the second takes two, the third keeps its own
    p = q4_ref.plan([40, 16, 5], [20, 16, 5], [4, 20, 3], [[7, 3, 9], [1, -1, -1], [4, -1, -1]],
                    [6, 2, 0, 5, 8, -7, -7, -7, -7, -7], 16, 30)
    assert p["table"] == [[7, 3, 9], [1, 9, 8], [4, -1, -1]]
    assert p["free"] == [6, 2, 0, 5] and p["cover_out"] == [24, 36, 8] and p["start"] == [0, 4, 24, 27]
    assert p["slot"][:5] == [3 * 16 + 4, 3 * 16 + 5, 3 * 16 + 6, 3 * 16 + 7, 9 * 16] and p["slot"][27:] == [-1] * 3
    assert p["pos"][4:24] == list(range(16, 36)) and p["slot"][20] == 8 * 16 and p["fault"] == 0
