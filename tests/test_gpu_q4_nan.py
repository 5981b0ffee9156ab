"""NaN in V reaches the queries that see it, all of them and no others, however
the work is split over blocks (kv_q4_attend against plain 64-bit attention)."""
import math

import pytest
import torch

from tests import q4_ref
from tests.test_gpu_q4_attend import build, call

pytestmark = pytest.mark.gpu


def poison(c, row, pos, head, block):
    """NaN in 16 dimensions of V of one position."""
    page, dh = c["kc"].shape[2], c["q"].shape[2]
    c["vc"][c["table"][row][pos // page], head, pos % page, dh // 2 + block] = 0x7F if pos % 2 else 0xFF


def check_nan(c, scale, calls=1, **kw):
    """NaN where the plain form has it; elsewhere the bounds of test_gpu_q4_attend. Returns where NaN is."""
    ref, rlse, spread, reach, flat = q4_ref.attend(c["q"].double(), c["kc"], c["vc"], c["table"], c["start"], c["length"],
                                                   scale, 0, c["k_exp"], c["v_exp"])
    wide, dh = c["q"].dtype == torch.float32, c["q"].shape[2]
    d = ((2.0 ** -21 if wide else 2.0 ** -16) + dh * 2.0 ** -24) * reach
    rel = 2 * d + 2.0 ** -21 + (2.0 ** -22 if wide else 2.0 ** -11)
    tol = ref.abs() * (2.0 ** -24 if wide else 2.0 ** -8) + rel[..., None] * spread * (1 + 2.0 ** -8) + 1e-30 + 2.0 ** -32 * flat
    nan = ref.isnan()
    for i in range(calls):
        out, lse, status = call(c, scale, **kw)
        assert status == 0
        lost, made = ~out.isnan() & nan, out.isnan() & ~nan
        assert not lost.any() and not made.any(), (i, int(lost.sum()), int(made.sum()), (lost | made).nonzero()[:5])
        assert ((out.double() - ref).abs() <= tol)[~nan].all(), i
        assert not lse.isnan().any()
    return nan


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh,group,hint", [(64, 1, 3), (64, 4, 40), (128, 2, 3), (128, 4, 40), (128, 4, 8), (256, 2, 3), (256, 4, 40)])
def test_blocks_with_many_one_tile_shares(dh, group, hint, dtype):
    """Rows of up to 128 positions: some seven shares of one tile each a block, so that V of a share is expanded while the
    notes of NaN of the shares before it are still to be read."""
    nkv, rows = 8, 130
    g = torch.Generator().manual_seed(dh + hint)
    q = (1 + torch.arange(rows) % 3).tolist()
    kv = [int(torch.randint(n, 129, (1,), generator=g)) for n in q]
    c = build(rows, q, kv, group * nkv, nkv, dh, 16, dtype, 7)
    for r in range(rows):
        if r % 4:
            for h in range(nkv):
                last = r % 4 == 3  # (the newest position: the row's last query alone sees it)
                poison(c, r, kv[r] - 1 if last else int(torch.randint(0, kv[r], (1,), generator=g)), h,
                       int(torch.randint(0, dh // 16, (1,), generator=g)))
    nan = check_nan(c, 1 / math.sqrt(dh), calls=3, max_q=hint)
    assert nan.any() and (~nan).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq,nkv,dh", [(4, 2, 64), (8, 2, 128), (24, 4, 256)])
@pytest.mark.parametrize("rows,kv", [(1, 300), (1, 2000), (1, 9000), (170, 300)])
def test_nan_of_no_weight_shows_however_the_row_is_split(rows, kv, nq, nkv, dh, dtype):
    """All weight of a row lies in its newest tile, 2^-200 of it and less elsewhere, and NaN in the oldest. By the formula
    0 x NaN is NaN: a block that sums both tiles shows it, and so has a join of several blocks' parts to."""
    c = build(rows, [2] * rows, [kv] * rows, nq, nkv, dh, 16, dtype, 33, exps=False)
    c["q"] = c["q"].abs() + 1
    for r in range(rows):
        for p in range(-(-kv // 16)):
            # codes 1.0 and one scale for all: the scores of a page are equal, 0 but on the last one
            c["kc"][c["table"][r][p], :, :, : dh // 2] = 0x22
            c["kc"][c["table"][r][p], :, : kv - 16 * p, dh // 2:] = q4_ref.e4m3_code(
                torch.tensor(16.0 if 16 * p + 16 >= kv else 0.0, dtype=torch.float64)).item()
        for h in range(nkv):
            poison(c, r, 5, h, h)
    # (16 sum q >= 16 dh, so that page's scores are 150 and more, 2^216 times the others' weight)
    nan = check_nan(c, 150 / (16 * dh))
    assert nan[:, :, :].any(-1).all() and (~nan).any()
