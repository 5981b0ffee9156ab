"""Plain 64-bit implementations of the paged 4-bit cache's operators and of the
log probabilities, for the tests (CPU, torch and Python; no library code)."""
from __future__ import annotations

import math

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
CAPACITY, BAD_ARG, NONFINITE = 1 << 8, 1 << 9, 1 << 10


# ------------------------------------------------------------------ page plans

def plan(cover, keep, new, table, free, page, max_tokens):
    """One plan on a Python stack. Returns a dict; 'free' holds the stack's entries only."""
    rows, max_pages, n_pages = len(cover), len(table[0]), len(free)
    table = [list(t) for t in table]
    start = [0]
    for n in new:
        start.append(start[-1] + max(n, 0))
    cap = page * max_pages
    clamp = [min(max(c, 0), cap) for c in cover]
    held = [-(-c // page) for c in clamp]
    stack = list(free[: max(0, n_pages - sum(held))])
    broken = n_pages < sum(held)
    fault, ok = 0, []
    for r in range(rows):
        bad = cover[r] != clamp[r] or keep[r] < 0 or keep[r] > cover[r] or new[r] < 0
        big = not bad and keep[r] + new[r] > cap
        late = start[r + 1] > max_tokens
        fault |= (BAD_ARG if bad or broken or late else 0) | (CAPACITY if big else 0)
        ok.append(not (bad or big or broken or late))
    want = [-(-(keep[r] + new[r]) // page) if ok[r] else held[r] for r in range(rows)]
    for r in reversed(range(rows)):
        for p in reversed(range(want[r], held[r])):
            stack.append(table[r][p])
    left, dry = len(stack), False
    for r in range(rows):
        if ok[r] and want[r] > held[r]:
            if dry or want[r] - held[r] > left:
                dry, ok[r], fault = True, False, fault | CAPACITY
                continue
            left -= want[r] - held[r]
            for p in range(held[r], want[r]):
                table[r][p] = stack.pop()
    slot, pos = [-1] * max_tokens, [-1] * max_tokens
    for r in range(rows):
        for i in range(max(new[r], 0)):
            t = start[r] + i
            if t >= max_tokens:
                break
            pos[t] = keep[r] + i
            if ok[r]:
                slot[t] = table[r][pos[t] // page] * page + pos[t] % page
    return dict(table=table, free=stack, cover_out=[keep[r] + new[r] if ok[r] else clamp[r] for r in range(rows)],
                start=[min(s, max_tokens) for s in start], slot=slot, pos=pos, fault=fault, ok=ok,
                pages=[want[r] if ok[r] else held[r] for r in range(rows)])


# ------------------------------------------------------------------ 4-bit rows

def e4m3_round(x):
    """To the nearest e4m3 value (ties to even, at most 448); x >= 0, float64."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def e4m3_code(v):
    """The byte of a value that e4m3 holds exactly (v >= 0)."""
    return v.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def quantize(x, exp=None):
    """x [T, H, dh] -> (bytes [T, H, dh*9/16] uint8, values float64). exp [H] ints."""
    y = x.to(torch.float64)
    if exp is not None:
        y = y * (2.0 ** -exp.to(torch.float64))[:, None]
    b = y.reshape(*y.shape[:-1], -1, 16)
    mag = b.abs()
    # the quotient is formed in fp32 by definition
    scale = e4m3_round((mag.amax(-1, keepdim=True).float() / 6).double())
    dist = (mag.unsqueeze(-1) - LEVELS * scale.unsqueeze(-1)).abs()
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: argmin keeps the first of equals
    code = order[dist[..., order].argmin(-1)]
    code = torch.where(scale > 0, code, 0)
    val = LEVELS[code] * scale * torch.where(b < 0, -1.0, 1.0)
    nib = (code + torch.where(torch.signbit(b) & (scale > 0), 8, 0)).to(torch.uint8).flatten(-2)
    raw = torch.cat([nib[..., 0::2] | (nib[..., 1::2] << 4), e4m3_code(scale.squeeze(-1))], -1)
    val = val.reshape(x.shape)
    if exp is not None:
        val = val * (2.0 ** exp.to(torch.float64))[:, None]
    return raw.contiguous(), val


def values(raw, dh):
    """float64 values [..., dh] of rows of bytes (head exponent 0)."""
    codes = raw[..., : dh // 2].long()
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = LEVELS[nib & 7] * torch.where(nib >= 8, -1.0, 1.0).double()
    s = raw[..., dh // 2:].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
    return v * s.repeat_interleave(16, -1)


# ------------------------------------------------------------------ attention

def attend(q, kc, vc, table, start, length, scale, window=0, k_exp=None, v_exp=None):
    """q [T, n_q, dh] float64; caches as bytes. Returns (out, lse, spread, reach, flat): spread = sum_j p_j |v_j|
    and flat = sum_j |v_j| per element, reach = scale * max_j sum_i |q_i k_ji| per query, the sizes that the
    tolerances go by."""
    T, nq, dh = q.shape
    nkv, page = kc.shape[1], kc.shape[2]
    G = nq // nkv
    out, spread, flat = (torch.zeros(T, nq, dh, dtype=torch.float64) for _ in range(3))
    lse = torch.full((T, nq), -math.inf, dtype=torch.float64)
    reach = torch.zeros(T, nq, dtype=torch.float64)
    for r in range(len(length)):
        a, b, n = start[r], start[r + 1], length[r]
        if a == b or n == 0:
            continue
        pages = torch.tensor([table[r][p] for p in range(-(-n // page))])
        for h in range(nkv):
            k, v = (values(c[pages, h].reshape(-1, c.shape[3])[:n], dh) * 2.0 ** (0 if e is None else int(e[h]))
                    for c, e in ((kc, k_exp), (vc, v_exp)))
            for i in range(a, b):
                pos = n - (b - a) + (i - a)
                lo = max(0, pos - window + 1) if window else 0
                if pos < lo:
                    continue
                kk, vv = k[lo:pos + 1], v[lo:pos + 1]
                qi = q[i, h * G:(h + 1) * G]
                s = qi @ kk.T * scale
                p = torch.softmax(s, -1)
                out[i, h * G:(h + 1) * G] = p @ vv
                spread[i, h * G:(h + 1) * G] = p @ vv.abs()
                flat[i, h * G:(h + 1) * G] = vv.abs().sum(0)
                lse[i, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
                reach[i, h * G:(h + 1) * G] = abs(scale) * (qi.abs() @ kk.abs().T).amax(-1)
    return out, lse, spread, reach, flat


# ------------------------------------------------------------------ log probabilities

def logprobs(x, tok, top):
    """x [n, V] float64, tok list. Returns (logprob, rank, entropy, top_id, top_lp)."""
    n, V = x.shape
    lp, rank, ent = [], [], []
    ids, lps = torch.full((n, top), -1, dtype=torch.int64), torch.full((n, top), -math.inf, dtype=torch.float64)
    for r in range(n):
        top_x = x[r].max()
        empty = top_x == -math.inf
        # from the maximum: a sum of lowest values would not hold log V beside them
        logp = x[r] if empty else (x[r] - top_x) - torch.log(torch.exp(x[r] - top_x).sum())
        p = logp.exp()
        ent.append(0.0 if empty else float(-(p * logp)[p > 0].sum()))
        t = tok[r]
        if t < 0 or t >= V:
            lp.append(0.0)
            rank.append(-1)
        else:
            lp.append(float(logp[t]))
            rank.append(int((x[r] > x[r, t]).sum() + (x[r, :t] == x[r, t]).sum()))
        order = torch.sort(x[r], descending=True, stable=True).indices[:top]
        order = order[x[r, order] > -math.inf]
        ids[r, : len(order)], lps[r, : len(order)] = order, logp[order]
    return (torch.tensor(lp, dtype=torch.float64), torch.tensor(rank), torch.tensor(ent, dtype=torch.float64), ids, lps)
