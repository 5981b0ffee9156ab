"""kv_attend_prompt with outputs and inputs at every 16-byte alignment that its contract takes: the same bits as with
tensors of their own, and nothing written beside the output."""
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests.test_gpu_prompt import call, make, parts

pytestmark = pytest.mark.gpu


def at(x, off):
    """x in a buffer of 77s, `off` elements behind a 256-byte border; the buffer."""
    flat = torch.full((x.numel() + 256,), 77.0, dtype=x.dtype, device="cuda")
    assert flat.data_ptr() % 256 == 0
    view = flat[off:off + x.numel()].view(x.shape)
    view.copy_(x)
    return view, flat


@pytest.mark.parametrize("nq,nkv,dh", [(4, 2, 64), (8, 2, 128), (6, 1, 256), (5, 5, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sixteens", [1, 2, 3])
@pytest.mark.parametrize("bad", [False, True])
def test_outputs_at_16_bytes(nq, nkv, dh, dtype, sixteens, bad):
    c = make([70, 0, 300, 1], nq, nkv, dh, dtype, 51)
    if bad:  # outputs that what was cleaned out of V is added to
        parts(c)[2][120, 0, 7] = math.inf
    scale = 1 / math.sqrt(dh)
    want, lse, status = call(c, scale)
    assert status == 0
    off = sixteens * 16 // want.element_size()
    (q, _), (k, _), (v, _) = (at(t.cuda(), off) for t in parts(c))
    out, flat = at(torch.zeros_like(want, device="cuda"), off)
    assert out.data_ptr() % 32 == (16 if sixteens % 2 else 0)
    ws, _ = at(torch.zeros(m.kv_attend_prompt_workspace_bytes(371, 4), dtype=torch.uint8, device="cuda"), 16)
    got_lse = torch.zeros(lse.shape, device="cuda")
    m.kv_attend_prompt(q, k, v, torch.tensor(c["start"], dtype=torch.int32, device="cuda"), out, ws, 300, scale=scale, lse=got_lse)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(got_lse.cpu(), lse)
    assert (flat[:off] == 77).all() and (flat[off + want.numel():] == 77).all()
