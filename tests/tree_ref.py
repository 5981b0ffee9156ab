"""Plain 64-bit implementations of the operators for trees of drafts, for whole
prompts and for the rotated append, for the tests (CPU, torch and Python; no
library code)."""
from __future__ import annotations

import math

import torch

from tests import q4_ref

BAD_ARG = 1 << 9


# ------------------------------------------------------------------ trees

def line(parent, i):
    """Node i and its ancestors, from i up; None where a parent is invalid."""
    up = []
    while i >= 0:
        up.append(i)
        p = parent[i]
        if p < -1 or p >= i:
            return None
        i = p
    return up


def plan(parents, length, window=0):
    """parents: a list per row. Returns (pos, masks as sets, status) of the packed nodes."""
    pos, masks, status = [], [], 0
    for par, L in zip(parents, length):
        n = len(par)
        for i in range(n):
            up = line(par, i) if n <= 128 and L >= n else None
            if up is None:
                status |= BAD_ARG
                pos.append(-1)
                masks.append(set())
            else:
                pos.append(L - n + len(up) - 1)
                masks.append(set(up[:window] if window else up))
    return pos, masks, status


def words(masks):
    """Sets of nodes as int32 [tokens, 4]."""
    out = torch.zeros((len(masks), 4), dtype=torch.int64)
    for t, s in enumerate(masks):
        for a in s:
            out[t, a // 32] |= 1 << (a % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def attend(q, kc, vc, table, start, length, masks, pos, scale, window=0, k_exp=None, v_exp=None):
    """As q4_ref.attend, for trees: masks are sets of nodes per packed query."""
    T, nq, dh = q.shape
    nkv, page = kc.shape[1], kc.shape[2]
    G = nq // nkv
    out, spread, flat = (torch.zeros(T, nq, dh, dtype=torch.float64) for _ in range(3))
    lse = torch.full((T, nq), -math.inf, dtype=torch.float64)
    reach = torch.zeros(T, nq, dtype=torch.float64)
    for r in range(len(length)):
        a, b, L = start[r], start[r + 1], length[r]
        n, base = b - a, L - (b - a)
        if n == 0 or L == 0:
            continue
        pages = torch.tensor([table[r][p] for p in range(-(-L // page))])
        for h in range(nkv):
            k, v = (q4_ref.values(c[pages, h].reshape(-1, c.shape[3])[:L], dh) * 2.0 ** (0 if e is None else int(e[h]))
                    for c, e in ((kc, k_exp), (vc, v_exp)))
            for i in range(a, b):
                lo = max(0, min(max(pos[i], base), L - 1) - window + 1) if window else 0
                at = torch.tensor(list(range(lo, max(base, 0))) + sorted(base + x for x in masks[i] if x < n and base + x >= 0), dtype=torch.long)
                if at.numel() == 0:
                    continue
                kk, vv, qi = k[at], v[at], q[i, h * G:(h + 1) * G]
                s = qi @ kk.T * scale
                p = torch.softmax(s, -1)
                rows = slice(h * G, (h + 1) * G)
                out[i, rows], spread[i, rows], flat[i, rows] = p @ vv, p @ vv.abs(), vv.abs().sum(0)
                lse[i, rows] = torch.logsumexp(s, -1)
                reach[i, rows] = abs(scale) * (qi.abs() @ kk.abs().T).amax(-1)
    return out, lse, spread, reach, flat


def commit(parents, toks, choices, length, max_path):
    """Per row: (path, committed tokens, keep)."""
    out = []
    for par, tok, choice, L in zip(parents, toks, choices, length):
        n = len(par)
        path = [0] if n else []
        while n and len(path) < max_path:
            nxt = [c for c in range(n) if 0 <= par[c] < c and par[c] == path[-1] and tok[c] == choice[path[-1]]]
            if not nxt:
                break
            path.append(nxt[0])
        out.append((path, [choice[i] for i in path], L - n + len(path)))
    return out


# ------------------------------------------------------------------ prompts

def prompt(q, k, v, start, scale, window=0):
    """q [T, n_q, dh], k, v [T, n_kv, dh] float64. Returns (out, lse, spread, reach)."""
    T, nq, dh = q.shape
    G = nq // k.shape[1]
    out, spread = torch.zeros_like(q), torch.zeros_like(q)
    lse, reach = torch.full((T, nq), -math.inf, dtype=torch.float64), torch.zeros(T, nq, dtype=torch.float64)
    for a, b in zip(start, start[1:]):
        if a == b:
            continue
        i = torch.arange(b - a)
        seen = i <= i[:, None]
        if window:
            seen &= i > i[:, None] - window
        for h in range(nq):
            s = (q[a:b, h] @ k[a:b, h // G].T * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, -1)
            vv = v[a:b, h // G]
            out[a:b, h], spread[a:b, h] = p @ vv, p @ vv.abs()
            lse[a:b, h] = torch.logsumexp(s, -1)
            reach[a:b, h] = abs(scale) * (q[a:b, h].abs() @ k[a:b, h // G].abs().T).masked_fill(~seen, 0).amax(-1)
    return out, lse, spread, reach


# ------------------------------------------------------------------ rotated rows

def turned(x, w, pos, rot, freq, eps):
    """(rows after the norm, rows after the rotation) of x [T, heads, dh] float64."""
    y = x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    z = y.clone()
    angle = pos.double()[:, None, None] * freq
    a, b = y[..., : rot // 2], y[..., rot // 2: rot]
    z[..., : rot // 2] = a * angle.cos() - b * angle.sin()
    z[..., rot // 2: rot] = b * angle.cos() + a * angle.sin()
    return y, z
