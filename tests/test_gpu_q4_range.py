"""kv_q4_append of finite values beyond fp32's range after the head's exponent: they saturate, and are no NaN."""
import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests.test_gpu_q4_cache import new_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_finite_values_saturate(dtype, dh):
    # y = x 2^64: the scale is the largest, 448, and a code is y / 448 rounded, at most 6
    x = torch.zeros(2, 1, dh, dtype=torch.float64)
    x[0, 0, :8] = torch.tensor([1e30, -3e38, 448.0 * 2.0 ** -64, -224.0 * 2.0 ** -64, 2.0 ** 64, -2.0 ** 63, 100.0 * 2.0 ** -64, 0.0])
    x[1, 0, 16:18] = torch.tensor([float("inf"), 1.0])
    x = x.to(dtype).cuda()
    exp = torch.tensor([-64], dtype=torch.int32, device="cuda")
    k, v, cache = new_cache(1, 1, 16, dh, exp, exp)
    slot = torch.arange(2, dtype=torch.int32, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    m.kv_q4_append(cache, x[:1], x[:1], slot[:1], status=status[:1])
    m.kv_q4_append(cache, x[1:], x[1:], slot[1:], status=status[1:])
    assert status.tolist() == [0, 1 << 10]
    for c in (k, v):
        row = c[0, 0, 0].cpu().tolist()
        codes = [n for b in row[:4] for n in (b & 15, b >> 4)]
        assert codes == [7, 15, 2, 9, 7, 15, 0, 0] and row[dh // 2] == 0x7E
        assert row[4:dh // 2] == [0] * (dh // 2 - 4) and row[dh // 2 + 1:] == [0] * (dh // 16 - 1)
        assert c[0, 0, 1, dh // 2 + 1] == 0x7F  # the infinity's 16 elements alone
    ko, vo = (torch.zeros(2, 1, dh, dtype=dtype, device="cuda") for _ in range(2))
    m.kv_q4_read(cache, slot, ko, vo)
    want = torch.tensor([6.0, -6.0, 1.0, -0.5, 6.0, -6.0, 0.0, 0.0], dtype=torch.float64) * 448 * 2.0 ** -64
    for o in (ko, vo):
        assert torch.equal(o[0, 0, :8].cpu().double(), want)
        assert o[1, 0].isnan().sum() == 16 and o[1, 0, 16:32].isnan().all()
