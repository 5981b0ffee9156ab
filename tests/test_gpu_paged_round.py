"""The paged 4-bit operators as a program uses them: speculative rounds commit
the tokens that decoding one by one does (block = chain at temperature 0,
"feat(inference): support the qwen3_5_mtp drafter" issue, Reproduction
instructions), and their log probabilities are the logits'."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("head_dim,n_q,n_kv", [(128, 8, 2), (64, 4, 2), (256, 6, 1)])
def test_rounds_commit_what_decoding_one_by_one_does(head_dim, n_q, n_kv):
    import paged_round as p
    target = p.Target(vocab=1031, hidden=256, n_q=n_q, n_kv=n_kv, head_dim=head_dim, seed=head_dim)
    first = torch.tensor([3, 14, 159, 265, 358], dtype=torch.int32, device="cuda")
    tokens, logprobs, counts = p.speculate(target, first, 30)
    plain = p.one_by_one(target, first, max(len(t) for t in tokens))
    for r, got in enumerate(tokens):
        assert got == plain[r][: len(got)], r
        assert len(got) == 30 + int(counts[:, r].sum())
        assert all(x <= 0 for x in logprobs[r])
    assert 0 < int(counts.sum()) < counts.numel() * 3  # some drafts were taken, some rejected
