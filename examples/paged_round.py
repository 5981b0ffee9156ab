"""Speculative rounds of a small target model over the paged 4-bit cache.

Each round appends a block of depth + 1 positions a row, attends it, verifies
the drafts and reports the committed tokens' log probabilities:

  kv_page_plan    pages, slots and positions of the block, from device lengths
  kv_q4_append    the block's K and V into their slots
  kv_q4_attend    the block's attention over the row's pages
  spec_verify     accepts a prefix of the drafts and commits one token more
  spec_logprobs   log probability, rank, entropy and alternatives of each

The accepted counts stay on the device: they make the next round's lengths, and
the next plan takes the pages of rejected positions back. The host reads nothing
between rounds.

The target is one attention layer with random weights and no trained
checkpoint; its drafts come from a copy that looks at the last token only. Its
own products are in 64 bits, so that a token's K and V do not depend on how many
tokens are in the call.

  python examples/paged_round.py [rounds]
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mtp_speculative_decoding_step_gb300 as m  # noqa: E402


class Target:
    """tokens -> logits: embedding, rotary q/k, attention over the cache, residual, head."""

    def __init__(self, vocab=2048, hidden=512, n_q=8, n_kv=2, head_dim=128, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.V, self.nq, self.nkv, self.dh = vocab, n_q, n_kv, head_dim
        mat = lambda *s: (torch.randn(s, generator=g, device=device) / math.sqrt(s[0])).to(torch.bfloat16)
        self.embed = torch.randn((vocab, hidden), generator=g, device=device).to(torch.bfloat16)
        self.qkv = mat(hidden, (n_q + 2 * n_kv) * head_dim)
        self.out = mat(n_q * head_dim, hidden)
        self.head = mat(hidden, vocab)

    def project(self, tok, pos):
        """q, k, v [tokens, heads, head_dim] of packed tokens at their positions, q and k rotated."""
        x = (self.embed[tok.long()].double() @ self.qkv.double()).to(torch.bfloat16).view(-1, self.nq + 2 * self.nkv, self.dh)
        half = self.dh // 2
        freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
        angle = pos.clamp(min=0).float()[:, None, None] * freq
        rot = x[:, : self.nq + self.nkv].float()
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1).to(torch.bfloat16)
        return rot[:, : self.nq], rot[:, self.nq:], x[:, self.nq + self.nkv:]

    def logits(self, tok, attended):
        x = self.embed[tok.long()].double() + attended.flatten(1).double() @ self.out.double()
        return (x @ self.head.double()).float()

    def guess(self, tok):
        """A draft: the token that the model without its attention would choose."""
        return (self.embed[tok.long()].double() @ self.head.double()).argmax(-1).to(torch.int32)


class PagedTarget:
    """The target with its pages: `block` runs packed blocks of equal size through it."""

    def __init__(self, target, rows, page=16, max_pages=32, block=4, device="cuda"):
        self.t, self.rows, self.page = target, rows, page
        self.n_pages = rows * max_pages
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
        shape = (self.n_pages, target.nkv, page, m.kv_q4_row_bytes(target.dh))
        self.cache = m.kv_q4_cache(*(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)))
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(self.n_pages, dtype=torch.int32, device=device)
        self.cover, self.cover_next, self.keep = i32(rows), i32(rows), i32(rows)
        self.new, self.start = torch.full((rows,), block, dtype=torch.int32, device=device), i32(rows + 1)
        self.slot, self.pos = i32(rows * block), i32(rows * block)
        self.status = i32(1)
        self.block_len = block
        self.q_out = torch.zeros((rows * block, target.nq, target.dh), dtype=torch.bfloat16, device=device)
        self.ws = torch.empty(m.kv_q4_attend_workspace_bytes(self.cache, target.nq, block, torch.bfloat16), dtype=torch.uint8,
                              device=device)

    def block(self, tok):
        """tok [rows, block] -> logits [rows, block, V]; the block's positions stay covered."""
        m.kv_page_plan(self.cover, self.keep, self.new, self.table, self.free, self.cover_next, self.start, self.slot,
                       self.pos, self.page, status=self.status)
        self.cover, self.cover_next = self.cover_next, self.cover
        q, k, v = self.t.project(tok.flatten(), self.pos)
        m.kv_q4_append(self.cache, k, v, self.slot, status=self.status)
        m.kv_q4_attend(self.cache, q, self.table, self.start, self.cover, self.q_out, self.ws, self.block_len,
                       scale=1.0 / math.sqrt(self.t.dh), status=self.status)
        return self.t.logits(tok.flatten(), self.q_out).view(self.rows, self.block_len, -1)


def speculate(target, first, rounds, depth=3, top=3):
    """Greedy speculative rounds from the tokens `first` [rows]. Returns the committed tokens per row, their log
    probabilities and the accepted counts [rounds, rows]."""
    rows, V = first.numel(), target.V
    run = PagedTarget(target, rows, block=depth + 1)
    dev = first.device
    params = m.sampling_array([dict(temperature=0.0)] * rows)
    u = torch.full((rows, depth + 1), 0.5, device=dev)
    vws = torch.empty(m.spec_verify_workspace_bytes(rows, depth, V), dtype=torch.uint8, device=dev)
    n = rows * (depth + 1)
    lws = torch.empty(m.spec_logprobs_workspace_bytes(n, V, top), dtype=torch.uint8, device=dev)
    tokens, logprobs, counts = [], [], []
    current = first
    for _ in range(rounds):
        draft = torch.empty((rows, depth), dtype=torch.int32, device=dev)
        last = current
        for i in range(depth):
            draft[:, i] = last = target.guess(last)
        logits = run.block(torch.cat([current[:, None], draft], 1)).contiguous()
        n_acc = torch.empty(rows, dtype=torch.int32, device=dev)
        out = torch.empty((rows, depth + 1), dtype=torch.int32, device=dev)
        m.spec_verify(logits, draft, params, u, n_acc, out, vws, status=run.status)
        lp, rank, entropy = torch.empty(n, device=dev), torch.empty(n, dtype=torch.int32, device=dev), torch.empty(n, device=dev)
        ids, lps = torch.empty((n, top), dtype=torch.int32, device=dev), torch.empty((n, top), device=dev)
        m.spec_logprobs(logits.view(n, V), out.view(n), lp, lws, rank=rank, entropy=entropy, top_id=ids, top_lp=lps,
                        status=run.status)
        run.keep = run.keep + n_acc + 1  # the current token and the accepted drafts
        current = out.gather(1, n_acc[:, None].long()).squeeze(1)
        tokens.append(out)
        logprobs.append(lp.view(rows, depth + 1))
        counts.append(n_acc)
    assert int(run.status) == 0, int(run.status)  # the one read, after the last round
    rows_out = [[int(t) for o in tokens for t in o[r].tolist() if t >= 0] for r in range(rows)]
    rows_lp = [[float(x) for o, l in zip(tokens, logprobs) for t, x in zip(o[r].tolist(), l[r].tolist()) if t >= 0] for r in range(rows)]
    return rows_out, rows_lp, torch.stack(counts)


def one_by_one(target, first, steps):
    """The same decoding without drafts: one token a step."""
    run = PagedTarget(target, first.numel(), block=1)
    tok, out = first, []
    for _ in range(steps):
        tok = run.block(tok[:, None])[:, 0].argmax(-1).to(torch.int32)
        run.keep = run.keep + 1
        out.append(tok)
    assert int(run.status) == 0
    return torch.stack(out, 1).tolist()


def main(rounds=12):
    target = Target()
    first = torch.tensor([3, 14, 159, 265], dtype=torch.int32, device="cuda")
    tokens, logprobs, counts = speculate(target, first, rounds)
    plain = one_by_one(target, first, max(len(t) for t in tokens))
    for r, (got, lp) in enumerate(zip(tokens, logprobs)):
        same = got == plain[r][: len(got)]
        print(f"row {r}: {len(got)} tokens in {rounds} rounds, mean log probability {sum(lp) / len(lp):.3f}, "
              f"same as one by one: {same}")
    print(f"accepted drafts a round: {float(counts.float().mean()):.2f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 12)
