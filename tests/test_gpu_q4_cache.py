"""kv_q4_append and kv_q4_read against the plain 64-bit rounding: bytes and values equal."""
import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref

pytestmark = pytest.mark.gpu


def new_cache(n_pages, nkv, page, dh, k_exp=None, v_exp=None, fill=0xAA):
    shape = (n_pages, nkv, page, dh * 9 // 16)
    k, v = (torch.full(shape, fill, dtype=torch.uint8, device="cuda") for _ in range(2))
    return k, v, m.kv_q4_cache(k, v, k_exp, v_exp)


def inputs(T, nkv, dh, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, nkv, dh), generator=g) * torch.exp(spread * torch.randn((nkv, dh), generator=g))
    x[0, 0, :16] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -0.0])
    x[-1, -1, 16:32] = 0.0       # a block of zeros
    x[-1, 0, 32:48] = 1e-5       # below the smallest scale
    x[0, -1, 48:64] *= 1e4       # beyond the largest
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,nkv,dh,page,layout", [
    (1, 1, 64, 16, "whole"), (3, 2, 128, 16, "whole"), (32, 4, 256, 64, "fused"), (77, 5, 64, 48, "fused"),
    (130, 3, 128, 32, "odd"), (515, 2, 256, 128, "heads first")])
def test_append_writes_the_reference_bytes(T, nkv, dh, page, layout, dtype):
    k, v = inputs(T, nkv, dh, dtype, 1), inputs(T, nkv, dh, dtype, 2)
    exps = torch.tensor([(3 * h) % 7 - 3 for h in range(nkv)], dtype=torch.int32)
    n_pages = -(-T // page) + 2
    kc, vc, cache = new_cache(n_pages, nkv, page, dh, exps.cuda(), (-exps).cuda())
    slot = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    if T > 3:
        slot[2] = -1
    if layout == "fused":  # a slice of one projection
        x = torch.zeros(T, 3 * nkv + 1, dh, dtype=dtype)
        x[:, nkv + 1:2 * nkv + 1], x[:, 2 * nkv + 1:] = k, v
        x = x.cuda()
        kd, vd = x[:, nkv + 1:2 * nkv + 1], x[:, 2 * nkv + 1:]
    elif layout == "odd":  # rows that start between 16-byte boundaries
        x = torch.zeros(2, T * nkv * (dh + 1) + 1, dtype=dtype, device="cuda")
        kd, vd = (x[i, 1:].view(T, nkv, dh + 1)[:, :, :dh] for i in range(2))
        kd.copy_(k)
        vd.copy_(v)
    elif layout == "heads first":
        kd, vd = (y.transpose(0, 1).contiguous().cuda().transpose(0, 1) for y in (k, v))
    else:
        kd, vd = k.cuda(), v.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_append(cache, kd, vd, slot.cuda(), status=status)
    ko, vo = (torch.full((T, nkv, dh), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    m.kv_q4_read(cache, slot.cuda(), ko, vo, status=status)
    assert int(status) == 0
    untouched = torch.ones(n_pages * page, dtype=torch.bool)
    untouched[slot[slot >= 0].long()] = False
    for x, c, e, o in ((k, kc, exps, ko), (v, vc, -exps, vo)):
        raw, val = q4_ref.quantize(x, e)
        by_slot = c.cpu().transpose(1, 2).reshape(n_pages * page, nkv, -1)
        live = slot >= 0
        assert torch.equal(by_slot[slot[live].long()], raw[live])
        assert (by_slot[untouched] == 0xAA).all()
        val[~live] = 0
        assert torch.equal(o.cpu().double(), val.to(dtype).double())
        assert torch.equal(val.to(dtype).double(), val)  # the values are exact in either type


def test_bf16_quotients_agree_with_the_comparisons():
    """bf16 input is rounded through a quotient, fp32 input by exact comparisons: the same bytes for the same values, at
    every scale, on every border, one bf16 step to either side of it, and over random values."""
    scales = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()  # every finite scale above 0
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    on = (scales[:, None] * borders).to(torch.bfloat16)
    bits = on.view(torch.int16)
    near = torch.stack([on, (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)], -1).flatten(1)  # [126, 21]
    top = (scales * 6).to(torch.bfloat16)[:, None]  # makes the block's scale
    rows = torch.cat([torch.cat([top, near[:, :15]], 1), torch.cat([top, near[:, 6:]], 1)], 1)  # two blocks of 16
    rows = torch.cat([rows, -rows], 1).reshape(126, 1, 64)
    g = torch.Generator().manual_seed(8)
    noise = (torch.randn((4096, 1, 64), generator=g) * torch.exp(3 * torch.randn((4096, 1, 1), generator=g))).to(torch.bfloat16)
    x = torch.cat([rows, noise]).cuda()
    T = x.shape[0]
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    got = []
    for y in (x, x.float()):
        k, v, cache = new_cache(-(-T // 16), 1, 16, 64)
        m.kv_q4_append(cache, y, y, slot)
        got.append((k, v))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    raw, _ = q4_ref.quantize(x[:126].cpu())
    assert torch.equal(got[0][0].cpu().reshape(-1, 1, 36)[:126], raw)


def test_nonfinite_blocks_read_back_as_nan_and_are_reported():
    k, v = inputs(4, 2, 64, torch.bfloat16, 3), inputs(4, 2, 64, torch.bfloat16, 4)
    k[1, 0, 5], v[2, 1, 63], v[3, 0, 16] = float("nan"), float("inf"), -float("inf")
    _, _, cache = new_cache(1, 2, 16, 64)
    slot = torch.arange(4, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_q4_append(cache, k.cuda(), v.cuda(), slot, status=status)
    assert int(status) == 1 << 10
    ko, vo = (torch.zeros(4, 2, 64, device="cuda") for _ in range(2))
    m.kv_q4_read(cache, slot, ko, vo)
    kn, vn = ko.isnan().cpu(), vo.isnan().cpu()
    assert kn.sum() == 16 and kn[1, 0, :16].all()
    assert vn.sum() == 32 and vn[2, 1, 48:].all() and vn[3, 0, 16:32].all()


@pytest.mark.parametrize("bad", [-2, 32, 2 ** 31 - 1, -2 ** 31])
def test_slots_outside_the_cache_are_skipped_and_reported(bad):
    kc, vc, cache = new_cache(2, 1, 16, 64)
    x = inputs(3, 1, 64, torch.float32, 5).cuda()
    slot = torch.tensor([4, bad, -1], dtype=torch.int32, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    m.kv_q4_append(cache, x, x, slot, status=status[:1])
    assert status.tolist() == [1 << 9, 0]
    assert int((kc != 0xAA).any(-1).sum()) == 1 and int((vc != 0xAA).any(-1).sum()) == 1
    o = torch.full((2, 3, 1, 64), 3.0, device="cuda")
    m.kv_q4_read(cache, slot, o[0], o[1], status=status[1:])
    assert status.tolist() == [1 << 9, 1 << 9] and (o[:, 1:] == 0).all()


def test_offsets_past_32_bits():
    """Rows behind the 4 GiB mark of a cache of 5.4 GB an array."""
    n_pages, nkv, page, dh = 9216, 4, 1024, 256
    shape = (n_pages, nkv, page, 144)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = m.kv_q4_cache(k, v)
    slots = [0, 4 * 1024 ** 3 // (144 * 4) + 12345, n_pages * page - 1]
    slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
    x = inputs(3, nkv, dh, torch.bfloat16, 6)
    m.kv_q4_append(cache, x.cuda(), x.cuda(), slot)
    raw, val = q4_ref.quantize(x)
    for i, s in enumerate(slots):
        assert torch.equal(k[s // page, :, s % page].cpu(), raw[i])
    o = torch.zeros(2, 3, nkv, dh, device="cuda")
    m.kv_q4_read(cache, slot, o[0], o[1])
    assert torch.equal(o[0].cpu().double(), val) and torch.equal(o[1].cpu().double(), val)
