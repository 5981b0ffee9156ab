"""spec_logprobs against the plain 64-bit implementation.

Whole numbers (ranks, ids) are equal. Bounds of the rest, for fp32 sums: every
exp is within 2^-21 of itself (2 ulp, and the rounding of x - m, |x - m| < 2^7
where exp is above 2^-180), a sum of V terms in a tree of at most 2^9 serial
additions adds 2^-15 at the worst, so log S is off by 2^-14 at most; x - m and
the final sums round to half a step of the result's size each. The entropy's
second sum has terms of at most |x - m| e^(x-m) <= 2^-1.4 times e^0's and is off by the same 2^-14
relative to sum |x - m| e^(x-m) / S <= log V."""
import math

import pytest
import torch

import mtp_speculative_decoding_step_gb300 as m
from tests import q4_ref

pytestmark = pytest.mark.gpu


def call(x, tok, top, **kw):
    n, V = x.shape
    d = dict(device="cuda")
    lp, ent = torch.full((n,), 9.0, **d), torch.full((n,), 9.0, **d)
    rank = torch.full((n,), -9, dtype=torch.int32, **d)
    ids, lps = torch.full((n, top), -9, dtype=torch.int32, **d), torch.full((n, top), 9.0, **d)
    ws = torch.empty(m.spec_logprobs_workspace_bytes(n, V, top), dtype=torch.uint8, **d)
    status = torch.zeros(1, dtype=torch.int32, **d)
    m.spec_logprobs(x, torch.tensor(tok, dtype=torch.int32, **d), lp, ws, rank=rank, entropy=ent, top_id=ids, top_lp=lps,
                    status=status, **kw)
    torch.cuda.synchronize()
    return [t.cpu() for t in (lp, rank, ent, ids, lps)] + [int(status)]


def check(x, tok, top, x_dev=None):
    lp, rank, ent, ids, lps, status = call(x.cuda() if x_dev is None else x_dev, tok, top)
    rlp, rrank, rent, rids, rlps = q4_ref.logprobs(x.double(), tok, top)
    assert status == 0
    assert torch.equal(rank.long(), rrank) and torch.equal(ids.long(), rids)
    V = x.shape[1]

    def near(got, want, tol):
        same = (got.double() == want) | ((got.double() - want).abs() <= tol)
        assert same.all(), (got[~same][:4], want[~same][:4])
    near(lp, rlp, 2.0 ** -14 + rlp.abs() * 2.0 ** -22)
    near(lps, rlps, 2.0 ** -14 + rlps.abs() * 2.0 ** -22)
    near(ent, rent, 2.0 ** -14 * (2 + math.log(V)))


def logits(n, V, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, V), generator=g) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,top", [
    (1, 1, 1), (2, 5, 8), (3, 31, 0), (4, 257, 64), (5, 1000, 5), (3, 4099, 20), (1, 32769, 64), (70, 2048, 8),
    (2, 152064, 20), (6, 152064, 5), (1100, 130, 3)])
def test_matches_the_plain_form(n, V, top, dtype):
    x = logits(n, V, dtype, n + V)
    g = torch.Generator().manual_seed(V)
    tok = torch.randint(0, V, (n,), generator=g).tolist()
    if n > 1:
        tok[1] = -1
    check(x, tok, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_masks_and_empty_rows(dtype):
    V, top = 5000, 64
    x = logits(9, V, dtype, 7)
    x[0] = 1.5                                        # every logit equal: ids ascending, entropy log V
    x[1] = -math.inf                                  # nothing left
    x[2] = -math.inf
    x[2, 4321] = -7.0                                 # one token left
    x[3, :4990] = -math.inf                           # fewer left than alternatives
    x[4] = torch.finfo(dtype).min                     # all at the type's lowest value
    x[5, 100:] = torch.finfo(dtype).min               # a mask of the lowest value
    x[6] = (torch.arange(V) % 3).to(dtype)            # thousands of ties at the top
    x[7] = torch.arange(V).to(dtype) / 100            # ascending: every element a new maximum
    x[8, ::2], x[8, 1::2] = 0.0, -0.0                 # signed zeros are equal
    check(x, [17, 5, 4321, 4995, 4999, 50, 2500, 3, 4998], top)


@pytest.mark.parametrize("keep,V,top", [(70, 152064, 64), (5000, 152064, 64), (5000, 152064, 7), (900, 40000, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sparse_masks(keep, V, top, dtype):
    """A grammar leaves a few tokens, strewn over the vocabulary: fewer in a part than there are alternatives."""
    g = torch.Generator().manual_seed(keep + V)
    x = torch.full((3, V), -math.inf, dtype=dtype)
    for r in range(3):
        at = torch.randperm(V, generator=g)[:keep]
        x[r, at] = (torch.randn(keep, generator=g) * 3).to(dtype)
    x[2] = torch.where(x[2] == -math.inf, x[2], 1.25)  # and all alike
    check(x, [int((x[r] > -math.inf).nonzero()[keep // 2]) for r in range(3)], top)


@pytest.mark.parametrize("top", [1, 20, 64])
def test_the_top_of_the_row_in_few_threads(top):
    """The largest logits at a stride of a thread's elements, and in one run of ids."""
    V = 100000
    x = logits(3, V, torch.float32, 31, scale=1.0)
    x[0, ::1024] = 50 + torch.arange(0, 98).float() / 7
    x[1, 40000:42500] = 60 - torch.arange(2500).float() / 100
    x[2] = -torch.arange(V).float() / 1000
    check(x, [1024, 41000, 99999], top)


def test_tokens_at_masked_places():
    x = logits(3, 300, torch.float32, 1)
    x[0, 10] = -math.inf
    x[1, 10] = torch.finfo(torch.float32).min
    lp, rank, _, _, _, status = call(x.cuda(), [10, 10, 299], 2)
    assert status == 0 and lp[0] == -math.inf and lp[1] == torch.finfo(torch.float32).min and rank[:2].tolist() == [299, 299]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nonfinite_logits_are_reported(bad):
    x = logits(3, 4100, torch.float32, 2)
    x[1, 4099] = bad
    *_, ids, _, status = call(x.cuda(), [0, 1, 2], 5)
    assert status == 1 << 10 and ((ids >= -1) & (ids < 4100)).all()


def test_token_ids_outside_the_vocabulary_are_reported():
    x = logits(3, 64, torch.float32, 3)
    lp, rank, _, _, _, status = call(x.cuda(), [64, -2, 5], 0)
    assert status == 1 << 9 and lp[:2].tolist() == [0, 0] and rank[:2].tolist() == [-1, -1] and rank[2] >= 0


@pytest.mark.parametrize("offset,stride", [(0, 5003), (1, 5001), (3, 5000), (4, 5004)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(offset, stride, dtype):
    n, V = 5, 4997
    x = logits(n, V, dtype, 11)
    buf = torch.full((offset + n * stride,), 99.0, dtype=dtype, device="cuda")
    view = buf[offset:].view(n, stride)[:, :V]
    view.copy_(x)
    check(x, [1, 2, 3, 4, 4996], 9, x_dev=view)


def test_outputs_left_out_and_a_graph():
    x = logits(4, 3001, torch.float32, 12).cuda()
    tok = torch.tensor([5, 6, 7, -1], dtype=torch.int32, device="cuda")
    ws = torch.empty(m.spec_logprobs_workspace_bytes(4, 3001, 0), dtype=torch.uint8, device="cuda")
    a, b = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    m.spec_logprobs(x, tok, a, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.spec_logprobs(x, tok, b, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and a[3] == 0


def test_runs_alike_twice():
    x = logits(40, 152064, torch.bfloat16, 13).cuda()
    tok = list(range(40))
    one, two = call(x, tok, 64), call(x, tok, 64)
    assert all(torch.equal(p, q) for p, q in zip(one[:-1], two[:-1]))


@pytest.mark.parametrize("n,V,dtype,top", [(40, 152064, torch.float32, 20), (300, 32769, torch.bfloat16, 8), (900, 5000, torch.float32, 64)])
def test_a_repeated_call_gives_the_same_bits(n, V, dtype, top):
    """Logits from HBM the first time, from L2 after that."""
    x = logits(n, V, dtype, V).cuda()
    tok = [(37 * i) % V for i in range(n)]
    first = call(x, tok, top)
    for _ in range(12):
        again = call(x, tok, top)
        assert all(torch.equal(a, b) for a, b in zip(first[:5], again[:5])) and again[5] == 0
