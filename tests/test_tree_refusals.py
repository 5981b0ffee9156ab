"""Refusals of the entry points for trees, prompts and the rotated append that
need no GPU (nothing is launched), the rotation's table, and the plain
implementations that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import tree_ref

FAKE, FAR = 0x10000000, 0x40000000  # never dereferenced; FAR from FAKE
BAD = 9


@pytest.fixture(scope="module")
def L():
    from mtp_speculative_decoding_step_gb300 import _build
    _build.build()
    return m.lib()


def _c(**kw):
    d = dict(k=FAKE, v=FAKE + (1 << 20), k_exp=None, v_exp=None, n_kv=2, head_dim=128, page=16, n_pages=8)
    d.update(kw)
    return m.Q4Cache(*[d[n] for n, _ in m.Q4Cache._fields_])


def _cache(**kw):
    return ctypes.byref(_c(**kw))


BAD_CACHES = [dict(k=None), dict(v=FAKE + 8), dict(head_dim=96), dict(n_kv=0), dict(page=24), dict(n_pages=0)]


# ------------------------------------------------------------------ rotation

def _rope_args(**kw):
    r = m.mtp_rope(64, 1e4)
    d = dict(stream=None, cache=_cache(), tokens=2, n_q=4, q=FAR, qt=512, qh=128, k=2 * FAR, kt=256, kh=128, v=3 * FAR, vt=256,
             vh=128, dtype=1, q_norm=None, k_norm=None, eps=1e-6, rope=ctypes.byref(r), pos=4 * FAR, slot=4 * FAR, q_out=5 * FAR,
             k_out=6 * FAR, status=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(n_q=0), dict(n_q=1025), dict(q=None), dict(k=None), dict(v=None), dict(pos=None),
                                dict(slot=None), dict(q_out=None), dict(dtype=2), dict(rope=None), dict(eps=-1.0), dict(eps=math.nan),
                                dict(eps=math.inf), dict(q=FAR + 1), dict(v=FAR + 1), dict(q_out=5 * FAR + 8), dict(k_out=6 * FAR + 2),
                                dict(q_norm=FAKE + 4), dict(k_norm=FAKE + 8), dict(tokens=1 << 29),
                                # overlaps: an output over another's input, over its own laid out otherwise, over the other output
                                dict(q_out=2 * FAR), dict(k_out=3 * FAR), dict(q_out=FAR, qt=520), dict(q_out=FAR + 16), dict(k_out=5 * FAR + 64),
                                dict(q=5 * FAR + 1024, qt=-512, q_out=5 * FAR),
                                # over what says where rows go, over the norms; strides that no memory has
                                dict(q_out=4 * FAR), dict(k_out=4 * FAR), dict(k_norm=6 * FAR), dict(q_norm=5 * FAR + 512),
                                dict(qt=1 << 62), dict(kh=-(1 << 61)), dict(tokens=3, vt=(1 << 63) - 4)])
def test_append_rope_refuses(L, kw):
    assert L.kv_q4_append_rope(*_rope_args(**kw)) == BAD


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_append_rope_refuses_a_bad_cache(L, kw):
    assert L.kv_q4_append_rope(*_rope_args(cache=_cache(**kw))) == BAD


@pytest.mark.parametrize("rot", [-2, 7, 130, 256])
def test_append_rope_refuses_a_bad_width(L, rot):
    r = m.Rope()
    r.rot_dim = rot
    assert L.kv_q4_append_rope(*_rope_args(rope=ctypes.byref(r))) == BAD


@pytest.mark.parametrize("rot,theta", [(-2, 1e4), (3, 1e4), (258, 1e4), (64, 0.0), (64, -1.0), (64, math.nan), (64, math.inf)])
def test_rope_refuses(L, rot, theta):
    with pytest.raises(m.MTPError):
        m.mtp_rope(rot, theta)


def test_rope_refuses_bad_frequencies(L):
    with pytest.raises(m.MTPError):
        m.mtp_rope(8, freq=[1.0, 2.0])
    with pytest.raises(m.MTPError):
        m.mtp_rope(4, freq=[1.0, math.nan])
    assert L.mtp_rope_init(4, 1e4, None, None) == BAD


@pytest.mark.parametrize("rot,theta", [(2, 1e4), (64, 1e6), (256, 1e7), (256, 1e4), (30, 2.5)])
def test_rope_table(L, rot, theta):
    """Turns a position: off by no more than 4 roundings of a double (pow, quotient, product of 2 pi's)."""
    r = m.mtp_rope(rot, theta)
    assert r.rot_dim == rot
    for i in range(rot // 2):
        want = theta ** (-2 * i / rot) / (2 * math.pi)
        assert abs(r.turn[i] / 2.0 ** 64 - want) <= 4 * 2.0 ** -53 * want + 2.0 ** -64


def test_rope_table_of_frequencies(L):
    r = m.mtp_rope(8, freq=[0.0, 2 * math.pi, -1.0, 7.0])
    got = [t / 2.0 ** 64 for t in r.turn[:4]]
    assert got[0] == 0 and min(got[1], 1 - got[1]) < 2.0 ** -52
    assert abs(got[2] - (1 - 1 / (2 * math.pi))) < 2.0 ** -50 and abs(got[3] - (7 / (2 * math.pi) - 1)) < 2.0 ** -50


# ------------------------------------------------------------------ trees

@pytest.mark.parametrize("at,val", [(1, 0), (1, 4097), (2, -1), (3, None), (4, None), (5, None), (6, -1), (7, None), (8, None),
                                    (8, 5 * FAR + 4), (7, FAKE), (7, 2 * FAR + 4), (7, 3 * FAR), (8, FAKE + 16), (8, 2 * FAR), (7, 5 * FAR + 16)])
def test_tree_plan_refuses(L, at, val):
    #       stream rows tokens parent start    len      window pos      mask     status
    args = [None, 2, 10, FAKE, 2 * FAR, 3 * FAR, 0, 4 * FAR, 5 * FAR, None]
    args[at] = val
    assert L.kv_tree_plan(*args) == BAD


@pytest.mark.parametrize("at,val", [
    (2, 0), (2, 4097), (3, 0), (3, 5), (4, -1), (5, None), (5, FAKE + 1), (8, 2), (9, None), (10, 0), (10, 1 << 28),
    (11, None), (12, None), (13, None), (13, FAKE + 4), (15, 0), (15, 129), (16, math.inf), (17, -1), (18, None), (18, FAKE + 8),
    (21, None), (21, FAKE + 4)])
def test_attend_tree_refuses(L, at, val):
    args = [None, _cache(), 1, 4, 1, FAKE, 512, 128, 1, FAKE, 4, FAKE, FAKE, FAKE, None, 1, 0.1, 0, FAKE, None, None, FAKE]
    args[at] = val
    assert L.kv_q4_attend_tree(*args) == BAD


def test_attend_tree_wants_positions_with_a_window(L):
    args = [None, _cache(), 1, 4, 1, FAKE, 512, 128, 1, FAKE, 4, FAKE, FAKE, FAKE, None, 1, 0.1, 7, FAKE, None, None, FAKE]
    assert L.kv_q4_attend_tree(*args) == BAD


def _commit_args(caches=None, **kw):
    arr = (m.Q4Cache * 2)(*(caches or [_c(), _c(k=FAKE + (2 << 20), v=FAKE + (3 << 20))]))
    d = dict(stream=None, caches=arr, n=2, rows=2, tokens=10, table=FAR, max_pages=4, start=2 * FAR, len=3 * FAR, parent=4 * FAR,
             tok=5 * FAR, choice=6 * FAR, max_path=5, n_acc=7 * FAR, out_tok=8 * FAR, keep=9 * FAR, path=10 * FAR, status=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw", [dict(caches=None), dict(n=-1), dict(n=65), dict(rows=0), dict(rows=4097), dict(tokens=-1), dict(table=None),
                                dict(max_pages=0), dict(max_pages=1 << 27), dict(start=None), dict(len=None), dict(parent=None),
                                dict(tok=None), dict(choice=None), dict(max_path=0), dict(max_path=129), dict(n_acc=None),
                                dict(out_tok=None), dict(keep=None),
                                dict(keep=3 * FAR), dict(n_acc=2 * FAR + 8), dict(out_tok=5 * FAR + 4), dict(path=6 * FAR), dict(path=8 * FAR + 36),
                                dict(keep=7 * FAR + 4), dict(out_tok=FAR + 28)])
def test_commit_refuses(L, kw):
    args = _commit_args(**{k: v for k, v in kw.items() if k != "caches"})
    if "caches" in kw:
        args[1] = None
    assert L.kv_q4_tree_commit(*args) == BAD


@pytest.mark.parametrize("second", [dict(k=None), dict(head_dim=64), dict(n_kv=4), dict(page=32), dict(n_pages=7), dict(k=FAKE), dict(v=FAKE + (1 << 20)),
                                    dict(k=FAKE + (1 << 20)), dict(k=FAKE + 16), dict(k=FAKE + 8 * 2 * 16 * 72 - 16)])
def test_commit_refuses_layers_of_other_shapes_or_the_same_twice(L, second):
    d = dict(k=FAKE + (2 << 20), v=FAKE + (3 << 20))
    d.update(second)
    assert L.kv_q4_tree_commit(*_commit_args([_c(), _c(**d)])) == BAD


# ------------------------------------------------------------------ prompts

def _prompt_args(**kw):
    d = dict(stream=None, rows=2, n_q=4, n_kv=2, dh=128, tokens=10, q=FAR, qt=512, qh=128, k=2 * FAR, kt=256, kh=128, v=3 * FAR, vt=256,
             vh=128, dtype=1, start=FAKE, max_len=5, scale=0.1, window=0, out=5 * FAR, lse=6 * FAR, status=None, ws=7 * FAR)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw", [dict(rows=0), dict(rows=4097), dict(n_q=0), dict(n_q=5), dict(n_q=1026), dict(n_kv=0), dict(dh=96), dict(dh=512),
                                dict(tokens=-1), dict(tokens=1 << 29), dict(q=None), dict(k=None), dict(v=None), dict(start=None), dict(out=None),
                                dict(ws=None), dict(dtype=2), dict(max_len=0), dict(scale=math.nan), dict(window=-1), dict(q=FAR + 8),
                                dict(k=2 * FAR + 2), dict(qt=516), dict(vh=132), dict(out=5 * FAR + 8), dict(ws=7 * FAR + 8), dict(out=FAR),
                                dict(out=2 * FAR + 512), dict(lse=3 * FAR), dict(q=5 * FAR + 9 * 1024, qt=-512),
                                # strides that the copies do not take, in either type
                                dict(qt=0), dict(kh=0), dict(vt=-256), dict(kt=0, dtype=0), dict(vh=-128, dtype=0), dict(qt=1 << 39), dict(kt=1 << 38, dtype=0),
                                dict(vt=1 << 62), dict(lse=6 * FAR + 2), dict(start=FAKE + 1), dict(out=FAKE - 1024), dict(lse=FAKE),
                                dict(lse=5 * FAR + 64)])
def test_prompt_refuses(L, kw):
    assert L.kv_attend_prompt(*_prompt_args(**kw)) == BAD


def test_prompt_workspace(L):
    assert m.kv_attend_prompt_workspace_bytes(100, 3) > 0
    assert [m.kv_attend_prompt_workspace_bytes(*a) for a in ((-1, 1), (5, 0), (5, 4097))] == [0] * 3


def test_nothing_to_do_is_not_an_error(L):
    r = m.mtp_rope(64)
    assert L.kv_q4_append_rope(None, _cache(), 0, 4, None, 0, 0, None, 0, 0, None, 0, 0, 1, None, None, 1e-6, ctypes.byref(r), None, None,
                               None, None, None) == 0
    assert L.kv_tree_plan(None, 1, 0, None, None, None, 0, None, None, None) == 0
    assert L.kv_q4_attend_tree(None, _cache(), 1, 4, 0, None, 0, 0, 1, None, 4, None, None, None, None, 1, 0.1, 0, None, None, None, None) == 0
    assert L.kv_attend_prompt(None, 1, 4, 2, 128, 0, None, 0, 0, None, 0, 0, None, 0, 0, 1, None, 1, 0.1, 0, None, None, None, None) == 0


def test_binding_refuses_wrong_shapes_and_types(L):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    c = m.kv_q4_cache(u8(4, 2, 16, 72), u8(4, 2, 16, 72))
    q, x, r = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128), m.mtp_rope(64)
    bad = []
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x, r, i32(2), i32(3), q.clone(), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x, r, i32(3), i32(3).long(), q.clone(), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x.bfloat16(), r, i32(3), i32(3), q.clone(), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x, r, i32(3), i32(3), q.half(), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x, r, i32(3), i32(3), q.clone(), q_norm=torch.zeros(64), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q, x, x, r, i32(3), i32(3), q.clone(), k_out=q.clone(), stream=0))
    bad.append(lambda: m.kv_q4_append_rope(c, q[..., :64], x, x, r, i32(3), i32(3), q[..., :64].clone(), stream=0))
    bad.append(lambda: m.kv_tree_plan(i32(3), i32(3), i32(2), i32(3), i32(3, 2), stream=0))
    bad.append(lambda: m.kv_tree_plan(i32(3), i32(2), i32(2), i32(3), i32(3, 4), stream=0))
    bad.append(lambda: m.kv_tree_plan(i32(3), i32(3), i32(2), i32(4), i32(3, 4), stream=0))
    ws = u8(1 << 26)
    bad.append(lambda: m.kv_q4_attend_tree(c, q, i32(1, 4), i32(2), i32(1), i32(3, 3), q.clone(), ws, 3, 1.0, stream=0))
    bad.append(lambda: m.kv_q4_attend_tree(c, q, i32(1, 4), i32(2), i32(1), i32(3, 4), q.clone(), ws[:16], 3, 1.0, stream=0))
    bad.append(lambda: m.kv_q4_attend_tree(c, q, i32(1, 4), i32(2), i32(1), i32(3, 4), q.clone(), ws, 3, 1.0, pos=i32(4), stream=0))
    cs = m.kv_q4_caches([c])
    ok = [cs, i32(2, 4), i32(3), i32(2), i32(5), i32(5), i32(5), i32(2), i32(2, 3), i32(2)]
    for at, wrong in ((1, i32(1, 4)), (2, i32(2)), (3, i32(3)), (5, i32(4)), (6, i32(5).long()), (7, i32(1)), (9, i32(3))):
        args = list(ok)
        args[at] = wrong
        bad.append(lambda args=args: m.kv_q4_tree_commit(*args, stream=0))
    bad.append(lambda: m.kv_q4_tree_commit(*ok, path=i32(2, 4), stream=0))
    bad.append(lambda: m.kv_attend_prompt(q, x, x[:2], i32(2), q.clone(), u8(64), 3, 1.0, stream=0))
    bad.append(lambda: m.kv_attend_prompt(q, x, x, i32(2), q.clone(), u8(0), 3, 1.0, stream=0))
    bad.append(lambda: m.kv_attend_prompt(q, x, x, i32(2).long(), q.clone(), ws, 3, 1.0, stream=0))
    bad.append(lambda: m.kv_attend_prompt(q, x, x, i32(2), q.bfloat16(), ws, 3, 1.0, stream=0))
    bad.append(lambda: m.kv_attend_prompt(q, x, x, i32(2), q.clone(), ws, 3, 1.0, lse=torch.zeros(3, 3), stream=0))
    for i, f in enumerate(bad):
        with pytest.raises(m.MTPError):
            f()
            pytest.fail(str(i))


# ------------------------------------------------------------------ the plain implementations

def test_ref_trees_worked_example():
    parents = [[-1, 0, 0, 1, 3, 2], [-1, -1, 0]]
    pos, masks, status = tree_ref.plan(parents, [16, 3])
    assert status == 0 and pos == [10, 11, 11, 12, 13, 12, 0, 0, 1]
    assert masks == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 3, 4}, {0, 2, 5}, {0}, {1}, {0, 2}]
    assert tree_ref.plan(parents, [16, 3], 2)[1][4] == {3, 4}
    pos, masks, status = tree_ref.plan([[-1, 1, 1, 0], [0]], [9, 0])
    assert status and pos == [5, -1, -1, 6, -1] and masks[2] == set() and masks[3] == {0, 3}
    assert tree_ref.words([{0, 33, 127}]).tolist() == [[1, 2, 0, -2 ** 31]]


def test_ref_commit_worked_example():
    (path, toks, keep), (p2, t2, k2) = tree_ref.commit([[-1, 0, 0, 2, 2, 4], []], [[9, 5, 6, 7, 8, 1], []], [[6, 0, 8, 0, 2, 0], []], [26, 4], 5)
    assert path == [0, 2, 4] and toks == [6, 8, 2] and keep == 23 and (p2, t2, k2) == ([], [], 4)
    assert tree_ref.commit([[-1, 0, 0]], [[9, 5, 5]], [[5, 1, 2]], [3], 5)[0][0] == [0, 1]  # the lower of two equal children
    assert tree_ref.commit([[-1, 0, 1]], [[9, 5, 5]], [[5, 5, 2]], [3], 2)[0][0] == [0, 1]  # cut


def test_ref_prompt_matches_pytorch():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((7, h, 16), generator=g, dtype=torch.float64) for h in (4, 2, 2))
    out, lse, *_ = tree_ref.prompt(q, k, v, [0, 3, 7], 0.3)
    for a, b in ((0, 3), (3, 7)):
        want = torch.nn.functional.scaled_dot_product_attention(q[a:b].transpose(0, 1), k[a:b].repeat_interleave(2, 1).transpose(0, 1),
                                                                v[a:b].repeat_interleave(2, 1).transpose(0, 1), is_causal=True, scale=0.3)
        assert torch.allclose(out[a:b].transpose(0, 1), want, atol=1e-12)
    one, *_ = tree_ref.prompt(q, k, v, [0, 7], 0.3, window=1)
    assert torch.allclose(one, v.repeat_interleave(2, 1))
