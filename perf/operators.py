"""Measured cases of the paged 4-bit cache operators and of the log probabilities.

Four operators that surround one speculative round of a target model:

  plan      pages, block tables and slot maps from the rows' lengths (kv_page_plan)
  append    K/V rows rounded to 4 bits into their slots, and read back (kv_q4_append, kv_q4_read)
  attend    attention of a block of queries per row over the paged 4-bit cache (kv_q4_attend)
  logprobs  log probabilities, ranks, entropy and alternatives of given tokens (spec_logprobs)

Where ``own`` is false each is computed in its plain form (elementary torch
operations in 32 bits); where it is true, by the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # pages of 8 sequences that each append a block of 4 (depth 3), after a verify that trimmed some drafts
        dict(name="plan 8 rows", op="plan", rows=8, page=64, max_pages=260, lo=1024, hi=16384, new_lo=4, new_hi=4, trim=3),
        # a large batch admitting prompts of odd lengths beside running rows
        dict(name="plan 512 rows prompts", op="plan", rows=512, page=16, max_pages=640, lo=0, hi=8191, new_lo=1, new_hi=1999, trim=40),
        # K/V of one verify block: 8 rows of 4 positions at the 27B heads
        dict(name="append block of 32", op="append", tokens=32, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", fused=True),
        # K/V of a prompt chunk, an odd count
        dict(name="append prompt 16383", op="append", tokens=16383, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", fused=True),
        # one sequence, depth 2: three queries over 4096 positions (the headline decoding shape)
        dict(name="attend 1 row block 3", op="attend", rows=1, q_lo=3, q_hi=3, lo=4096, hi=4096, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", window=0),
        # the batched workload: 8 ragged rows of 1k-16k, depth 3
        dict(name="attend 8 rows block 4", op="attend", rows=8, q_lo=4, q_hi=4, lo=1024, hi=16384, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", window=0),
        # 64 rows of plain decoding (single tokens) with odd lengths, small pages, the reduced head shape
        dict(name="attend 64 rows single", op="attend", rows=64, q_lo=1, q_hi=1, lo=1, hi=16383, n_q=8, n_kv=2, dh=128, page=16, dtype="bf16", window=0),
        # prompt chunks behind a long prefix: up to 2048 queries at offsets near 8192
        dict(name="attend prompt 2 rows", op="attend", rows=2, q_lo=1500, q_hi=2048, lo=8192, hi=10240, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", window=0),
        # the tiny fp32 head with a sliding window
        dict(name="attend tiny fp32 window", op="attend", rows=3, q_lo=1, q_hi=5, lo=67, hi=1000, n_q=4, n_kv=2, dh=64, page=32, dtype="f32", window=333),
        # log probabilities of one row's verified block (depth 2)
        dict(name="logprobs 3 of 152064", op="logprobs", n=3, V=152064, top=5, dtype="f32"),
        # 64 rows of depth 3
        dict(name="logprobs 256 of 152064", op="logprobs", n=256, V=152064, top=20, dtype="f32"),
        # an odd vocabulary in bf16 (many equal logits), many positions
        dict(name="logprobs 1001 of 32769 bf16", op="logprobs", n=1001, V=32769, top=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "logprobs", "logprobs"])
    if op == "plan":
        rows, page = _log(rng, 1, 512), rng.choice([16, 32, 48, 64, 128])
        hi, new_hi = _log(rng, 16, 8191), _log(rng, 1, 1999)
        return dict(op=op, rows=rows, page=page, max_pages=-(-(hi + new_hi) // page) + 1, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, trim=rng.randint(0, 40))
    n_q, n_kv, dh = rng.choice([(24, 4, 256), (8, 2, 128), (4, 2, 64), (8, 8, 128), (16, 2, 256), (5, 5, 64)])
    page, dtype = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16383), n_q=n_q, n_kv=n_kv, dh=dh, page=page, dtype=dtype, fused=rng.random() < 0.5)
    if op == "attend":
        rows = _log(rng, 1, 64)
        q_hi = _log(rng, 1, 17) if rng.random() < 0.7 else _log(rng, 17, 1500)
        hi = _log(rng, 16, 16384)
        while rows * q_hi * n_q * hi > 2 * 2048 * 24 * 10240 or rows * n_kv * dh * hi > 8 * 4 * 256 * 16384:
            rows, hi = max(1, rows // 2), max(16, hi * 3 // 4)
        q_hi = min(q_hi, hi)
        return dict(op=op, rows=rows, q_lo=rng.randint(1, q_hi), q_hi=q_hi, lo=rng.randint(1, hi), hi=hi, n_q=n_q, n_kv=n_kv, dh=dh,
                    page=page, dtype=dtype, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    V = _log(rng, 129, 152064)
    return dict(op=op, n=_log(rng, 1, max(1, min(1500, 256 * 152064 // V))), V=V, top=rng.choice([0, 1, 5, 8, 20, 64]),
                dtype=rng.choice(["f32", "f32", "bf16"]))


def _spread(lo, hi, n):
    """n whole numbers of [lo, hi], evenly strewn, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]


def _lens(case):
    """Query counts and cache lengths of an attend case's rows (no more queries than positions)."""
    q, kv = _spread(case["q_lo"], case["q_hi"], case["rows"]), _spread(case["lo"], case["hi"], case["rows"])[::-1]
    return [min(a, b) for a, b in zip(q, kv)], kv


def _visible(case):
    """(query, key) pairs that the mask leaves, and the cache slots that some query of their row sees."""
    pairs = slots = 0
    w = case["window"] or 1 << 40
    for a, b in zip(*_lens(case)):
        for i in ((0, a - 1) if a > 1 else (0,)):
            assert b - a + i >= 0
        n = [min(w, b - a + i + 1) for i in range(a)]
        pairs += sum(n)
        slots += min(b, w + a - 1)
    return pairs, slots


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "buf": {}}
    if case["op"] == "plan":
        n, page, mp = case["rows"], case["page"], case["max_pages"]
        keep = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        trim = torch.randint(0, case["trim"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["keep"], s["cover"] = keep, torch.clamp(keep + trim, max=page * mp)
        s["new"] = torch.randint(case["new_lo"], case["new_hi"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["n_pages"] = n * mp
        perm = torch.randperm(n * mp, generator=g, device=DEV).to(torch.int32)
        held = (s["cover"] + page - 1) // page
        at = (torch.cumsum(held, 0) - held)[:, None] + torch.arange(mp, device=DEV)
        inside = torch.arange(mp, device=DEV) < held[:, None]
        s["table"] = torch.where(inside, perm[at.clamp(max=n * mp - 1)], -1).to(torch.int32).contiguous()
        s["free"] = torch.roll(perm, -int(held.sum()))
        s["max_tokens"] = n * case["new_hi"]
        for name, size in (("cover_out", n), ("start", n + 1), ("slot", s["max_tokens"]), ("pos", s["max_tokens"])):
            s[name] = torch.zeros(size, dtype=torch.int32, device=DEV)
    elif case["op"] == "append":
        t, nq, nkv, dh, page = (case[k] for k in ("tokens", "n_q", "n_kv", "dh", "page"))
        dt = DT[case["dtype"]]
        x = torch.randn((t, nq + 2 * nkv, dh), generator=g, device=DEV)
        x *= torch.exp(0.7 * torch.randn((nq + 2 * nkv, dh), generator=g, device=DEV))  # channels of unlike size
        x = x.to(dt)
        s["k"], s["v"] = x[:, nq:nq + nkv], x[:, nq + nkv:]
        if not case["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        s["n_pages"] = -(-t // page) + 3
        slot = torch.randperm(s["n_pages"] * page, generator=g, device=DEV)[:t].to(torch.int32)
        slot[torch.rand(t, generator=g, device=DEV) < 0.01] = -1  # padding
        s["slot"] = slot
        s["k_exp"] = torch.randint(-3, 4, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        s["v_exp"] = torch.randint(-3, 4, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        shape = (s["n_pages"], nkv, page, dh * 9 // 16)
        s["kc"], s["vc"] = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
        s["k_out"], s["v_out"] = (torch.zeros((t, nkv, dh), dtype=dt, device=DEV) for _ in range(2))
    elif case["op"] == "attend":
        nq, nkv, dh, page = (case[k] for k in ("n_q", "n_kv", "dh", "page"))
        dt = DT[case["dtype"]]
        ql, kl = _lens(case)
        mp = -(-max(kl) // page)
        pages = [-(-b // page) for b in kl]
        n_pages = sum(pages) + 2
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        at = [sum(pages[:r]) for r in range(len(pages))]
        idx = _rows(at)[:, None] + torch.arange(mp, device=DEV)
        inside = torch.arange(mp, device=DEV) < _rows(pages)[:, None]
        s["table"] = torch.where(inside, perm[idx.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
        s["kc"] = _pack(torch.randn((n_pages, nkv, page, dh), generator=g, device=DEV))
        s["vc"] = _pack(torch.randn((n_pages, nkv, page, dh), generator=g, device=DEV))
        s["k_exp"] = torch.randint(-1, 2, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        s["v_exp"] = torch.randint(-3, 4, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        t = sum(ql)
        s["q"] = (1.5 * torch.randn((t, nq, dh), generator=g, device=DEV)).to(dt)
        s["start"] = _rows([sum(ql[:r]) for r in range(len(ql) + 1)])
        s["len"] = _rows(kl)
        s["max_q"], s["max_kv"] = max(ql), max(kl)
        s["scale"] = 1.0 / math.sqrt(dh)
        s["out"] = torch.zeros((t, nq, dh), dtype=dt, device=DEV)
        s["lse"] = torch.zeros((t, nq), dtype=torch.float32, device=DEV)
    else:
        n, V, top = case["n"], case["V"], case["top"]
        x = torch.randn((n, V), generator=g, device=DEV) * 2.5
        peak = torch.randint(0, V, (n, 3), generator=g, device=DEV)
        x.scatter_add_(1, peak, 12.0 * torch.rand((n, 3), generator=g, device=DEV))  # a few likely tokens a row
        x[:, V - V // 100:] = -math.inf  # ids past the tokenizer's
        x[::5, : V // 3] = torch.finfo(torch.float32).min  # a grammar's mask on some rows
        s["logits"] = x.to(DT[case["dtype"]]) if case["dtype"] == "f32" else _lowest(x.to(torch.bfloat16))
        tok = torch.where(torch.rand(n, generator=g, device=DEV) < 0.6, peak[:, 0],
                          torch.randint(0, V, (n,), generator=g, device=DEV)).to(torch.int32)
        tok %= V - V // 100
        tok[::5] = V // 3 + tok[::5] % (V - V // 100 - V // 3)  # a grammar lets none of its masked tokens through
        tok[torch.rand(n, generator=g, device=DEV) < 0.05] = -1  # past a row's committed tokens
        s["tok"] = tok
        for name in ("logprob", "entropy"):
            s[name] = torch.zeros(n, device=DEV)
        s["rank"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        s["top_id"] = torch.zeros((n, top), dtype=torch.int32, device=DEV)
        s["top_lp"] = torch.zeros((n, top), device=DEV)
    return s


def _lowest(x):
    """The bf16 type's lowest value where rounding float32's lowest gave -inf, below the vocabulary's padding."""
    V = x.shape[1]
    x[::5, : V // 3] = torch.finfo(torch.bfloat16).min
    return x


# ------------------------------------------------------------------ the 4-bit format, plain

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _round4(y):
    """(codes 0..7, negative, scale) of blocks of 16 along the last dimension, as [..., dh/16, 16] and [..., dh/16, 1]."""
    b = y.unflatten(-1, (-1, 16))
    mag = b.abs()
    scale = (mag.amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    code = ((mag > 0.25 * scale).to(torch.uint8) + (mag >= 0.75 * scale) + (mag > 1.25 * scale) + (mag >= 1.75 * scale)
            + (mag > 2.5 * scale) + (mag >= 3.5 * scale) + (mag > 5.0 * scale))
    return torch.where(scale > 0, code, 0), b < 0, scale


def _pack(y):
    """Cache rows of values [..., dh]: dh/2 bytes of codes (the even element in the low half), then dh/16 scales."""
    code, neg, scale = _round4(y)
    nib = (code + 8 * neg).to(torch.uint8).flatten(-2)
    return torch.cat([nib[..., 0::2] | (nib[..., 1::2] << 4), scale.squeeze(-1).to(torch.float8_e4m3fn).view(torch.uint8)], -1).contiguous()


def _unpack(raw, dh):
    """float32 values [..., dh] of cache rows."""
    lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=raw.device)
    codes = raw[..., : dh // 2]
    val = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (val.unflatten(-1, (-1, 16)) * raw[..., dh // 2:].contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


# ------------------------------------------------------------------ one pass

def run(state):
    return {"plan": _plan, "append": _append, "attend": _attend, "logprobs": _logprobs}[state["case"]["op"]](state)


def _plan(s):
    page = s["case"]["page"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        m.kv_page_plan(s["cover"], s["keep"], s["new"], s["table"], s["free"], s["cover_out"], s["start"], s["slot"], s["pos"], page)
        return {k: s[k] for k in ("table", "free", "cover_out", "start", "slot", "pos")}
    cover, keep, new, table, free = s["cover"], s["keep"], s["new"], s["table"], s["free"]
    mp, n_pages, T = table.shape[1], free.shape[0], s["slot"].shape[0]
    held, total = (cover + page - 1) // page, keep + new
    want = (total + page - 1) // page
    rel, take = (held - want).clamp(min=0), (want - held).clamp(min=0)
    R, K = torch.cumsum(rel, 0) - rel, torch.cumsum(take, 0) - take
    top = n_pages - held.sum() + rel.sum()
    granted = (K + take <= top) | (take == 0)
    taken = torch.where(granted, take, 0).sum()
    start = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)]).to(torch.int32)
    p = torch.arange(mp, device=DEV)[None]
    given = (p >= want[:, None]) & (p < held[:, None])
    at = torch.where(given, top - 1 - (R[:, None] + p - want[:, None]), n_pages)
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at.flatten(), table.flatten())[:n_pages]
    got = (p >= held[:, None]) & (p < want[:, None]) & granted[:, None]
    table = torch.where(got, stack[(top - 1 - (K[:, None] + p - held[:, None])).clamp(0, n_pages - 1)], table)
    free = torch.where(torch.arange(n_pages, device=DEV) < top - taken, stack, free)
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(start[1:].contiguous(), t.int(), right=True, out_int32=True).clamp(max=cover.shape[0] - 1)
    live = t < start[-1]
    pos = keep[row] + t - start[row]
    slot = table[row, (pos // page).clamp(0, mp - 1)] * page + pos % page
    slot = torch.where(live & granted[row], slot, -1).to(torch.int32)
    return {"table": table, "free": free, "cover_out": torch.where(granted, total, cover), "start": start, "slot": slot,
            "pos": torch.where(live, pos, -1).to(torch.int32)}


def _append(s):
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        c = s["buf"].get("cache") or s["buf"].setdefault("cache", m.kv_q4_cache(s["kc"], s["vc"], s["k_exp"], s["v_exp"]))
        m.kv_q4_append(c, s["k"], s["v"], s["slot"])
        m.kv_q4_read(c, s["slot"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    out = {}
    live = (s["slot"] >= 0)[:, None, None]
    lut = torch.tensor(_E2M1, device=DEV)
    for name in ("k", "v"):
        x = s[name].float()
        exp = s[name + "_exp"].float()[:, None]
        code, neg, scale = _round4(x * torch.exp2(-exp))
        val = (lut[code.int()] * torch.where(neg, -scale, scale)).flatten(-2) * torch.exp2(exp)
        out[name] = torch.where(live, val, 0.0).to(s[name].dtype)
    return out


def _attend(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            b["cache"] = m.kv_q4_cache(s["kc"], s["vc"], s["k_exp"], s["v_exp"])
            b["ws"] = torch.empty(m.kv_q4_attend_workspace_bytes(b["cache"], c["n_q"], s["max_q"], s["q"].dtype), dtype=torch.uint8, device=DEV)
        m.kv_q4_attend(b["cache"], s["q"], s["table"], s["start"], s["len"], s["out"], b["ws"], s["max_q"], scale=s["scale"],
                       window=c["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    nq, nkv, dh, page, R = c["n_q"], c["n_kv"], c["dh"], c["page"], c["rows"]
    G, Q, L = nq // nkv, s["max_q"], s["max_kv"]
    q_len = s["start"][1:] - s["start"][:-1]
    l = torch.arange(L, device=DEV)
    pages = s["table"][:, l // page].clamp(min=0)

    def cached(cache, exp):  # [R, nkv, L, dh]
        val = _unpack(cache[pages, :, l % page], dh)
        return (val * torch.exp2(exp.float())[:, None]).transpose(1, 2)

    i = torch.arange(Q, device=DEV)
    at = (s["start"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().unflatten(2, (nkv, G)).permute(0, 2, 1, 3, 4).reshape(R, nkv, Q * G, dh)
    sc = torch.matmul(q, cached(s["kc"], s["k_exp"]).transpose(2, 3)).unflatten(2, (Q, G)) * s["scale"]
    here = (s["len"] - q_len)[:, None] + i
    seen = (l <= here[..., None]) & (l < s["len"][:, None, None])
    if c["window"]:
        seen &= l > here[..., None] - c["window"]
    sc.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m_ = sc.amax(-1, keepdim=True)
    m_ = torch.where(m_ == -math.inf, 0.0, m_)
    p = torch.exp(sc.sub_(m_))
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), cached(s["vc"], s["v_exp"])).unflatten(2, (Q, G)) / torch.where(tot > 0, tot, 1.0)
    lse = (m_ + torch.log(tot)).squeeze(-1)
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    row = torch.searchsorted(s["start"][1:].contiguous(), t, right=True)
    col = t - s["start"][row]
    return {"out": o[row, :, col].flatten(1, 2).to(s["q"].dtype), "lse": lse[row, :, col].flatten(1, 2)}


def _logprobs(s):
    top = s["case"]["top"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            n, V = s["logits"].shape
            b["ws"] = torch.empty(m.spec_logprobs_workspace_bytes(n, V, top), dtype=torch.uint8, device=DEV)
        m.spec_logprobs(s["logits"], s["tok"], s["logprob"], b["ws"], rank=s["rank"], entropy=s["entropy"], top_id=s["top_id"], top_lp=s["top_lp"])
        return {k: s[k] for k in ("logprob", "rank", "entropy", "top_id", "top_lp")}
    x, tok = s["logits"].float(), s["tok"].long()
    n, V = x.shape
    m_ = x.amax(1, keepdim=True)
    d = x - m_
    e = torch.exp(d)
    tot = e.sum(1, keepdim=True)
    log = torch.log(tot)
    entropy = (log - torch.where(e > 0, d * e, 0.0).sum(1, keepdim=True) / tot).squeeze(1)
    live = tok >= 0
    xt = x.gather(1, tok.clamp(min=0)[:, None])
    ids = torch.arange(V, device=DEV)
    rank = ((x > xt) | ((x == xt) & (ids < tok[:, None]))).sum(1)
    out = {"logprob": torch.where(live, (xt - m_ - log).squeeze(1), 0.0), "rank": torch.where(live, rank, -1).to(torch.int32), "entropy": entropy}
    bits = (x + 0.0).view(torch.int32).long()
    key = (torch.where(bits < 0, -2147483648 - bits, bits) << 32) + (V - 1 - ids)  # the larger logit, then the lower id
    best = torch.topk(key, min(top, V), dim=1).values
    out["top_id"] = (V - 1 - (best & 0xFFFFFFFF)).to(torch.int32)
    out["top_lp"] = x.gather(1, out["top_id"].long()) - m_ - log
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "plan":
        n, page = case["rows"], case["page"]
        moved = n * (case["new_lo"] + case["new_hi"]) / 2 / page  # pages taken: read from the stack, written to the table
        return {"bytes": 4 * (3 * n + 2 * n + 1 + 2 * moved + 2 * n * case["new_hi"]), "flops": 0}
    if case["op"] == "append":
        values = 2 * case["tokens"] * case["n_kv"] * case["dh"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": values * (size + 9 / 16) + values * (size + 9 / 16) + 8 * case["tokens"], "flops": 0}
    if case["op"] == "attend":
        pairs, slots = _visible(case)
        size = 2 if case["dtype"] == "bf16" else 4
        q = sum(_lens(case)[0]) * case["n_q"]
        return {"bytes": slots * case["n_kv"] * 2 * case["dh"] * 9 // 16 + q * (2 * case["dh"] * size + 4),
                "flops": 4 * case["dh"] * case["n_q"] * pairs}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["n"] * (case["V"] * size + 16 + 8 * case["top"]), "flops": 0}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The outputs from the definitions in 64 bits, one row (or position) at a time; whole numbers have none."""
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "append":
        return {k: _exact_round(s[k], s[k + "_exp"], s["slot"]) for k in ("k", "v")}
    if case["op"] == "attend":
        return _exact_attend(s)
    x, tok = s["logits"].double(), s["tok"].tolist()
    lp, ent, tops = [], [], []
    for r, t in enumerate(tok):
        z = torch.logsumexp(x[r], 0)
        logp = x[r] - z
        lp.append(logp[t] if t >= 0 else z * 0)
        p = logp.exp()
        ent.append(-(p * logp)[p > 0].sum())
        order = torch.sort(x[r], descending=True, stable=True).values[: case["top"]]
        tops.append(order - z)
    return {"logprob": torch.stack(lp), "rank": None, "entropy": torch.stack(ent), "top_id": None, "top_lp": torch.stack(tops)}


def _exact_round(x, exp, slot):
    """The value of {0, .5, 1, 1.5, 2, 3, 4, 6} x block scale nearest to each element; an even code where two are as near."""
    y = x.double() * (2.0 ** -exp.double())[:, None]
    y = y.reshape(*y.shape[:-1], -1, 16)
    a = y.abs().amax(-1, keepdim=True) / 6
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)  # e4m3: four significant bits, 2^-9 apart at the least
    scale = (torch.round(a / step) * step).clamp(max=448.0)
    levels = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    best, at = None, None
    for code in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be strictly nearer
        off = (y.abs() - levels[code] * scale).abs()
        if best is None:
            best, at = off, torch.zeros_like(y)
        else:
            nearer = off < best
            best, at = torch.where(nearer, off, best), torch.where(nearer, levels[code], at)
    val = (torch.sign(y) * at * scale).reshape(x.shape) * (2.0 ** exp.double())[:, None]
    val[slot < 0] = 0
    return val


def _exact_attend(s):
    c = s["case"]
    nq, nkv, dh, page = c["n_q"], c["n_kv"], c["dh"], c["page"]
    G = nq // nkv
    out = torch.zeros((s["q"].shape[0], nq, dh), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["q"].shape[0], nq), dtype=torch.float64, device=DEV)
    start, length = s["start"].tolist(), s["len"].tolist()
    table = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=DEV)

    def values(cache, row, h, exp):  # [L, dh]
        n = length[row]
        pages = s["table"][row, : -(-n // page)].long()
        raw = cache[pages, h].reshape(-1, dh * 9 // 16)[:n]
        byte = raw[:, : dh // 2].long()
        nib = torch.empty((n, dh), dtype=torch.int64, device=DEV)
        nib[:, 0::2], nib[:, 1::2] = byte % 16, byte // 16
        scale = raw[:, dh // 2:].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
        return table[nib % 8] * sign[nib // 8] * scale.repeat_interleave(16, 1) * 2.0 ** int(exp[h])

    for r in range(c["rows"]):
        a, b, n = start[r], start[r + 1], length[r]
        if a == b:
            continue
        here = torch.arange(n - (b - a), n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        seen = key <= here
        if c["window"]:
            seen &= key > here - c["window"]
        for h in range(nkv):
            k, v = values(s["kc"], r, h, s["k_exp"]), values(s["vc"], r, h, s["v_exp"])
            for j in range(h * G, h * G + G):
                sc = (s["q"][a:b, j].double() @ k.T) * s["scale"]
                sc[~seen] = -math.inf
                lse[a:b, j] = torch.logsumexp(sc, 1)
                out[a:b, j] = torch.softmax(sc, 1) @ v
    return {"out": out, "lse": lse}
