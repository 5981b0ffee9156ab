"""The operators for trees as a program uses them: a prompt through the rotated
append and the prompt's attention, then rounds of tree drafts, commit the tokens
that decoding one by one does."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("head_dim,n_q,n_kv,rot", [(128, 8, 2, 64), (64, 4, 2, 64), (256, 6, 1, 64), (64, 3, 3, 22)])
def test_rounds_commit_what_decoding_one_by_one_does(head_dim, n_q, n_kv, rot):
    import tree_round as p
    target = p.Target(vocab=1031, hidden=256, n_q=n_q, n_kv=n_kv, head_dim=head_dim, rot=rot, seed=head_dim)
    prompts = [[(7 * i + r) % 1031 for i in range(n)] for r, n in enumerate((1, 130, 17, 64, 33))]
    tokens, counts = p.generate(target, prompts, 20)
    plain, _ = p.generate(target, prompts, max(len(t) for t in tokens), tree=[-1])
    for r, got in enumerate(tokens):
        assert got == plain[r][: len(got)], r
        assert len(got) == 21 + int(counts[:, r].sum())
    assert 0 < int(counts.sum())  # some drafts were taken
    assert int((counts == 0).sum()) > 0 or int((counts < 5).sum()) > 0  # and some rejected
