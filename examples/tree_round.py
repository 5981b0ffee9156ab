"""Speculative rounds that draft trees, over the paged 4-bit cache.

A prompt, then rounds of a small target model:

  kv_q4_append_rope   norms and rotation of the projection's rows, K and V into their slots
  kv_attend_prompt    the prompt's attention over its own unrounded K and V
and per round
  kv_page_plan        pages and slots of the tree's nodes, from device lengths
  kv_tree_plan        the nodes' positions and which of them see which
  kv_q4_append_rope   the nodes' rows, rotated by their positions
  kv_q4_attend_tree   each node over the committed positions and its ancestors
  spec_logprobs       the target's choice behind every node
  kv_q4_tree_commit   the path of nodes that the choices follow, its rows moved together

The confirmed lengths stay on the device and make the next round's plan. The target
is one attention layer with random weights and no trained checkpoint; its drafts
are the likeliest tokens by a look at the last token only.

  python examples/tree_round.py [rounds]
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

# node 0 is the last committed token; two drafts behind it, two behind the first of them, and so on down the likelier side
TREE = [-1, 0, 0, 1, 1, 2, 3, 3, 4, 6, 6, 9]


class Target:
    """tokens -> logits: embedding, normed and rotated q and k, attention, residual, head."""

    def __init__(self, vocab=2048, hidden=512, n_q=8, n_kv=2, head_dim=128, rot=64, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.V, self.nq, self.nkv, self.dh = vocab, n_q, n_kv, head_dim
        mat = lambda *s: (torch.randn(s, generator=g, device=device) / math.sqrt(s[0])).to(torch.bfloat16)
        self.embed = torch.randn((vocab, hidden), generator=g, device=device).to(torch.bfloat16)
        self.qkv, self.out, self.head = mat(hidden, (n_q + 2 * n_kv) * head_dim), mat(n_q * head_dim, hidden), mat(hidden, vocab)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device) for _ in range(2))
        self.rope = m.mtp_rope(rot, 1e6)

    def project(self, tok):
        """q, k, v of packed tokens: slices of one fused projection."""
        x = (self.embed[tok.long()].double() @ self.qkv.double()).to(torch.bfloat16).view(-1, self.nq + 2 * self.nkv, self.dh)
        return x[:, : self.nq], x[:, self.nq:self.nq + self.nkv], x[:, self.nq + self.nkv:]

    def logits(self, tok, attended):
        x = self.embed[tok.long()].double() + attended.flatten(1).double() @ self.out.double()
        return (x @ self.head.double()).float()

    def guesses(self, tok, count):
        """The tokens that the model without its attention would choose, the likeliest first."""
        return (self.embed[tok.long()].double() @ self.head.double()).topk(count, -1).indices.to(torch.int32)


class TreeTarget:
    """The target with its pages, for rounds of one tree shape."""

    def __init__(self, target, rows, tree=TREE, page=16, max_pages=32, device="cuda"):
        self.t, self.rows, self.tree, self.page, self.n = target, rows, tree, page, len(tree)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
        shape = (rows * max_pages, target.nkv, page, m.kv_q4_row_bytes(target.dh))
        self.cache = m.kv_q4_cache(*(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)))
        self.caches = m.kv_q4_caches([self.cache])
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(rows * max_pages, dtype=torch.int32, device=device)
        self.cover, self.cover_next, self.keep, self.start, self.status = i32(rows), i32(rows), i32(rows), i32(rows + 1), i32(1)
        self.parent = torch.tensor(tree * rows, dtype=torch.int32, device=device)
        self.scale = 1.0 / math.sqrt(target.dh)

    def _plan(self, new, tokens):
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=self.table.device)
        slot, pos = i32(tokens), i32(tokens)
        m.kv_page_plan(self.cover, self.keep, new, self.table, self.free, self.cover_next, self.start, slot, pos, self.page, status=self.status)
        self.cover, self.cover_next = self.cover_next, self.cover
        return slot, pos

    def _append(self, tok, pos, slot):
        q, k, v = self.t.project(tok)
        q_out, k_out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k, memory_format=torch.contiguous_format)
        m.kv_q4_append_rope(self.cache, q, k, v, self.t.rope, pos, slot, q_out, k_out=k_out, q_norm=self.t.q_norm, k_norm=self.t.k_norm,
                            status=self.status)
        return q_out, k_out, v

    def prompt(self, prompts):
        """The first token behind each prompt (lists of tokens, packed without padding)."""
        dev = self.table.device
        tok = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
        new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        slot, pos = self._plan(new, tok.numel())
        q, k, v = self._append(tok, pos, slot)
        out = torch.empty_like(q)
        ws = torch.empty(m.kv_attend_prompt_workspace_bytes(tok.numel(), self.rows), dtype=torch.uint8, device=dev)
        m.kv_attend_prompt(q, k, v, self.start, out, ws, max(len(p) for p in prompts), scale=self.scale, status=self.status)
        self.keep = self.cover.clone()
        last = self.start[1:].long() - 1
        return self.t.logits(tok[last], out[last]).argmax(-1).to(torch.int32)

    def draft(self, current):
        """Tokens [rows, nodes]: every node's children are its token's likeliest followers, in order."""
        tok = torch.zeros((self.rows, self.n), dtype=torch.int32, device=current.device)
        tok[:, 0] = current
        for i in range(self.n):
            kids = [c for c in range(self.n) if self.tree[c] == i and c > 0]
            if kids:
                tok[:, kids] = self.t.guesses(tok[:, i], len(kids))
        return tok

    def round(self, current):
        """One round behind the tokens `current` [rows]: (committed tokens [rows, nodes], -1 behind the last; accepted drafts [rows])."""
        dev, n, T = current.device, self.n, self.rows * self.n
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        tok = self.draft(current)
        slot, _ = self._plan(torch.full((self.rows,), n, dtype=torch.int32, device=dev), T)
        pos, mask = i32(T), i32(T, m.MTP_TREE_MAX // 32)
        m.kv_tree_plan(self.parent, self.start, self.cover, pos, mask, status=self.status)
        q, _, _ = self._append(tok.flatten(), pos, slot)
        out = torch.empty_like(q)
        ws = torch.empty(m.kv_q4_attend_workspace_bytes(self.cache, self.t.nq, n, q.dtype), dtype=torch.uint8, device=dev)
        m.kv_q4_attend_tree(self.cache, q, self.table, self.start, self.cover, mask, out, ws, n, scale=self.scale, status=self.status)
        logits = self.t.logits(tok.flatten(), out)
        choice, lp, top = i32(T, 1), torch.empty(T, device=dev), torch.empty((T, 1), device=dev)
        lws = torch.empty(m.spec_logprobs_workspace_bytes(T, self.t.V, 1), dtype=torch.uint8, device=dev)
        m.spec_logprobs(logits, torch.full((T,), -1, dtype=torch.int32, device=dev), lp, lws, top_id=choice, top_lp=top, status=self.status)
        n_acc, committed, keep = i32(self.rows), i32(self.rows, n), i32(self.rows)
        m.kv_q4_tree_commit(self.caches, self.table, self.start, self.cover, self.parent, tok.flatten(), choice.flatten(), n_acc, committed, keep,
                            status=self.status)
        self.keep = keep
        return committed, n_acc


def generate(target, prompts, rounds, tree=TREE):
    """Greedy rounds behind the prompts. Returns the generated tokens per row and the accepted counts [rounds, rows]."""
    run = TreeTarget(target, len(prompts), tree)
    current = run.prompt(prompts)
    out, counts = [current[:, None]], []
    for _ in range(rounds):
        committed, n_acc = run.round(current)
        current = committed.gather(1, n_acc[:, None].long()).squeeze(1)
        out.append(committed)
        counts.append(n_acc)
    assert int(run.status) == 0, int(run.status)  # the one read, after the last round
    return [[int(t) for o in out for t in o[r].tolist() if t >= 0] for r in range(len(prompts))], torch.stack(counts)


def main(rounds=12):
    target = Target()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, target.V, (n,), generator=g).tolist() for n in (5, 40, 1, 77)]
    tokens, counts = generate(target, prompts, rounds)
    plain, _ = generate(target, prompts, max(len(t) for t in tokens), tree=[-1])  # a tree of the root alone: one token a round
    for r, got in enumerate(tokens):
        print(f"row {r}: {len(got)} tokens in {rounds} rounds, same as one by one: {got == plain[r][: len(got)]}")
    print(f"accepted drafts a round: {float(counts.float().mean()):.2f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 12)
