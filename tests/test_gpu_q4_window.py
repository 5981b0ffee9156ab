"""Windows as large as the type holds ("no limit") give what no window gives, also for rows with more queries than
cached positions."""
import math

import pytest
import torch

from tests.test_gpu_q4_attend import HEADS, build, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nkv,dh", HEADS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 2 ** 30])
def test_the_largest_windows(nq, nkv, dh, dtype, window):
    c = build(5, [5, 40, 2, 130, 3], [2, 10, 300, 128, 0], nq, nkv, dh, 16, dtype, 31)
    out, lse = check(c, 1 / math.sqrt(dh), window)
    plain, plain_lse = check(c, 1 / math.sqrt(dh))
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
