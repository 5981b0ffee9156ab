"""Measured cases of the operators for tree drafts and for whole prompts.

Five operators of a target model's attention layer, from the projection's rows
to the committed cache, where a round drafts a tree instead of a chain:

  rope     per-head norms of queries and keys, the rotation by position, and the
           append of K and V to the paged 4-bit cache (kv_q4_append_rope)
  prompt   causal attention of whole packed prompts over unrounded K and V
           (kv_attend_prompt)
  plan     positions and ancestor masks of trees from their parents (kv_tree_plan)
  tree     attention of a tree's nodes over the cache and their ancestors
           (kv_q4_attend_tree)
  commit   the path that the target confirms, and its rows moved together in
           every layer's cache (kv_q4_tree_commit)

Where ``own`` is false each is computed in its plain form (elementary torch
operations in 32 bits, angles in 64); where it is true, by the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST = 128  # nodes of a tree
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one block of 8 rows of 4 positions at the 27B heads, rotated over the whole head as the drafter's own layer is
        dict(name="rope block of 32", op="rope", tokens=32, n_q=24, n_kv=4, dh=256, rot=256, theta=1e6, far=16384, page=64, dtype="bf16", norm=True),
        # a prompt chunk of an odd count, a quarter of each head rotated, far positions, K also given unrounded
        dict(name="rope prompt 16383", op="rope", tokens=16383, n_q=24, n_kv=4, dh=256, rot=64, theta=1e7, far=262144, page=64, dtype="bf16", norm=True),
        # two whole prompts of the 27B heads
        dict(name="prompt 2 rows 8k", op="prompt", rows=2, lo=5001, hi=8192, n_q=24, n_kv=4, dh=256, dtype="bf16", window=0),
        # a batch of ragged prompts at the reduced head shape
        dict(name="prompt 32 rows ragged", op="prompt", rows=32, lo=1, hi=2047, n_q=8, n_kv=2, dh=128, dtype="bf16", window=0),
        # the tiny fp32 head
        dict(name="prompt tiny fp32", op="prompt", rows=3, lo=5, hi=131, n_q=4, n_kv=2, dh=64, dtype="f32", window=0),
        # trees of 8 rows, 16 nodes each
        dict(name="plan 8 trees of 16", op="plan", rows=8, n_lo=16, n_hi=16, hi=16384, window=0, roots=0.0),
        # a large batch of trees of all sizes, in a window that is shorter than some of their paths
        dict(name="plan 512 trees", op="plan", rows=512, n_lo=1, n_hi=128, hi=16384, window=9, roots=0.05),
        # one sequence, a tree of 16 nodes over 4096 positions
        dict(name="tree 1 row of 16", op="tree", rows=1, q_lo=16, q_hi=16, lo=4096, hi=4096, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", window=0),
        # 8 ragged rows of 1k-16k, trees of up to 33 nodes
        dict(name="tree 8 rows of 33", op="tree", rows=8, q_lo=20, q_hi=33, lo=1024, hi=16384, n_q=24, n_kv=4, dh=256, page=64, dtype="bf16", window=0),
        # the tiny fp32 head with a sliding window, trees of odd sizes
        dict(name="tree tiny fp32 window", op="tree", rows=3, q_lo=1, q_hi=21, lo=67, hi=1000, n_q=4, n_kv=2, dh=64, page=32, dtype="f32", window=333),
        # a round's end for 8 rows: one layer
        dict(name="commit 8 rows 1 layer", op="commit", rows=8, n_lo=16, n_hi=16, hi=512, layers=1, n_kv=4, dh=256, page=64, max_path=9),
        # and for 64 rows: the 16 full-attention layers of the target
        dict(name="commit 64 rows 16 layers", op="commit", rows=64, n_lo=8, n_hi=64, hi=512, layers=16, n_kv=4, dh=256, page=16, max_path=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(24, 4, 256), (8, 2, 128), (4, 2, 64), (8, 8, 128), (16, 2, 256), (5, 5, 64)]


def draw(rng):
    op = rng.choice(["rope", "rope", "prompt", "prompt", "plan", "tree", "tree", "commit"])
    n_q, n_kv, dh = rng.choice(HEADS)
    page, dtype = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 16383), n_q=n_q, n_kv=n_kv, dh=dh, rot=rng.choice([0, 16, dh // 4, dh // 2, dh - 2, dh, dh]),
                    theta=rng.choice([1e4, 1e6, 1e7]), far=_log(rng, 2, 1048576), page=page, dtype=dtype, norm=rng.random() < 0.7)
    if op == "prompt":
        rows, hi = _log(rng, 1, 64), _log(rng, 1, 8192)
        most = 2 * 24 * 8192 ** 2 if dtype == "bf16" else 24 * 1024 ** 2
        while rows * n_q * hi * hi > most:
            rows, hi = max(1, rows // 2), max(1, hi * 3 // 4)
        return dict(op=op, rows=rows, lo=rng.randint(0, hi - 1), hi=hi, n_q=n_q, n_kv=n_kv, dh=dh, dtype=dtype, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    if op == "plan":
        n_hi = _log(rng, 1, MOST)
        return dict(op=op, rows=_log(rng, 1, 512), n_lo=rng.randint(0, n_hi), n_hi=n_hi, hi=_log(rng, 128, 1000000), window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    roots=rng.choice([0.0, 0.1]))
    if op == "commit":
        n_hi = _log(rng, 1, MOST)
        return dict(op=op, rows=_log(rng, 1, 64), n_lo=rng.randint(1, n_hi), n_hi=n_hi, hi=rng.randint(n_hi, 512), layers=_log(rng, 1, 16), n_kv=n_kv, dh=dh,
                    page=page, max_path=rng.randint(1, 24))
    rows, q_hi, hi = _log(rng, 1, 64), _log(rng, 1, MOST), _log(rng, 16, 16384)
    while rows * q_hi * n_q * hi > 32 * 33 * 24 * 16384 or rows * n_kv * dh * hi > 16 * 4 * 256 * 16384:
        rows, hi = max(1, rows // 2), max(16, hi * 3 // 4)
    q_hi = min(q_hi, hi)
    return dict(op=op, rows=rows, q_lo=rng.randint(1, q_hi), q_hi=q_hi, lo=rng.randint(1, hi), hi=hi, n_q=n_q, n_kv=n_kv, dh=dh, page=page, dtype=dtype,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]))


def _spread(lo, hi, n):
    """n whole numbers of [lo, hi], evenly strewn, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]


def _trees(case):
    """Node counts and cache lengths (the nodes among them) of a plan or commit case's rows."""
    n = _spread(case["n_lo"], case["n_hi"], case["rows"])
    return n, [max(a, b) for a, b in zip(n, _spread(case["hi"] // 2, case["hi"], case["rows"])[::-1])]


def _lens(case):
    """Node counts and cache lengths of a tree attention case's rows (no more nodes than positions)."""
    q, kv = _spread(case["q_lo"], case["q_hi"], case["rows"]), _spread(case["lo"], case["hi"], case["rows"])[::-1]
    return [min(a, b) for a, b in zip(q, kv)], kv


def _prompts(case):
    n = _spread(case["lo"], case["hi"], case["rows"])
    n[0] = case["hi"]
    return n


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(n):
    return _rows([sum(n[:r]) for r in range(len(n) + 1)])


def _parents(g, n, roots):
    """Parents of packed trees: node 0 is the root; a later one hangs below its forerunner or any earlier node, a share of them on nothing."""
    if sum(n) == 0:
        return _rows([])
    i = torch.cat([torch.arange(a, device=DEV) for a in n])
    u = torch.rand((3, i.numel()), generator=g, device=DEV)
    any_ = (u[0] * i).long().clamp(max=(i - 1).clamp(min=0))
    parent = torch.where(u[1] < 0.5, i - 1, any_)
    parent[(i == 0) | (u[2] < roots)] = -1
    return parent.to(torch.int32)


def _table(g, kl, page):
    """Block table of rows of these lengths, over strewn pages, and the number of pages."""
    mp = max(1, -(-max(kl) // page))
    pages = [-(-b // page) for b in kl]
    n_pages = sum(pages) + 2
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    idx = _rows([sum(pages[:r]) for r in range(len(pages))])[:, None] + torch.arange(mp, device=DEV)
    inside = torch.arange(mp, device=DEV) < _rows(pages)[:, None]
    return torch.where(inside, perm[idx.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous(), n_pages


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "buf": {}}
    if case["op"] == "rope":
        t, nq, nkv, dh, page = (case[k] for k in ("tokens", "n_q", "n_kv", "dh", "page"))
        dt = DT[case["dtype"]]
        x = torch.randn((t, nq + 2 * nkv, dh), generator=g, device=DEV)
        x *= torch.exp(0.7 * torch.randn((nq + 2 * nkv, dh), generator=g, device=DEV))  # channels of unlike size
        x = x.to(dt)
        s["q"], s["k"], s["v"] = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
        for name in ("q_norm", "k_norm"):
            s[name] = 1.0 + 0.1 * torch.randn(dh, generator=g, device=DEV) if case["norm"] else None
        s["n_pages"] = -(-t // page) + 3
        s["slot"] = torch.randperm(s["n_pages"] * page, generator=g, device=DEV)[:t].to(torch.int32)
        s["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
        pad = torch.rand(t, generator=g, device=DEV) < 0.01  # behind the last position of a padded batch
        s["slot"][pad] = -1
        s["pos"][pad] = -1
        s["k_exp"] = torch.randint(-3, 1, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        s["v_exp"] = torch.randint(-3, 4, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        shape = (s["n_pages"], nkv, page, dh * 9 // 16)
        s["kc"], s["vc"] = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
        s["q_out"] = torch.zeros((t, nq, dh), dtype=dt, device=DEV)
        s["k_out"] = torch.zeros((t, nkv, dh), dtype=dt, device=DEV)
        s["k_held"], s["v_held"] = (torch.zeros((t, nkv, dh), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    elif case["op"] == "prompt":
        nq, nkv, dh = (case[k] for k in ("n_q", "n_kv", "dh"))
        dt, n = DT[case["dtype"]], _prompts(case)
        t = sum(n)
        x = torch.randn((t, nq + 2 * nkv, dh), generator=g, device=DEV)
        x[:, :nq] *= 1.5  # (queries: sharper scores than 1 / sqrt(dh) leaves)
        x = x.to(dt)
        s["q"], s["k"], s["v"] = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
        s["start"], s["max_len"], s["scale"] = _starts(n), max(n), 1.0 / math.sqrt(dh)
        s["out"] = torch.zeros((t, nq, dh), dtype=dt, device=DEV)
        s["lse"] = torch.zeros((t, nq), dtype=torch.float32, device=DEV)
    elif case["op"] == "plan":
        n, kl = _trees(case)
        s["parent"], s["start"], s["len"] = _parents(g, n, case["roots"]), _starts(n), _rows(kl)
        s["pos"] = torch.zeros(sum(n), dtype=torch.int32, device=DEV)
        s["mask"] = torch.zeros((sum(n), MOST // 32), dtype=torch.int32, device=DEV)
    elif case["op"] == "commit":
        n, kl = _trees(case)
        s["parent"], s["start"], s["len"] = _parents(g, n, 0.0), _starts(n), _rows(kl)
        t, R, nkv, dh, page = sum(n), case["rows"], case["n_kv"], case["dh"], case["page"]
        s["tok"] = torch.randint(0, 4000, (t,), generator=g, device=DEV, dtype=torch.int32)
        s["choice"] = torch.randint(0, 4000, (t,), generator=g, device=DEV, dtype=torch.int32)
        # most nodes' target token is that of one of their children, so that paths are long
        row = torch.repeat_interleave(torch.arange(R, device=DEV), _rows(n).long())
        at = s["start"][row].long() + s["parent"]
        child = (s["parent"] >= 0) & (torch.rand(t, generator=g, device=DEV) < 0.8)
        first = torch.full((t,), t, device=DEV).scatter_reduce(0, at[child], torch.arange(t, device=DEV)[child], "amin")
        s["choice"] = torch.where(first < t, s["tok"][first.clamp(max=t - 1)], s["choice"])
        s["table"], s["n_pages"] = _table(g, kl, page)
        shape = (case["layers"], 2, s["n_pages"], nkv, page, dh * 9 // 16)
        s["kv"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        for name, size in (("n_acc", (R,)), ("keep", (R,)), ("out_tok", (R, case["max_path"])), ("path", (R, case["max_path"]))):
            s[name] = torch.zeros(size, dtype=torch.int32, device=DEV)
    else:
        nq, nkv, dh, page = (case[k] for k in ("n_q", "n_kv", "dh", "page"))
        dt = DT[case["dtype"]]
        ql, kl = _lens(case)
        s["table"], n_pages = _table(g, kl, page)
        s["kc"] = _pack(torch.randn((n_pages, nkv, page, dh), generator=g, device=DEV))
        s["vc"] = _pack(torch.randn((n_pages, nkv, page, dh), generator=g, device=DEV))
        s["k_exp"] = torch.randint(-1, 2, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        s["v_exp"] = torch.randint(-3, 4, (nkv,), generator=g, device=DEV, dtype=torch.int32)
        t = sum(ql)
        s["q"] = (1.5 * torch.randn((t, nq, dh), generator=g, device=DEV)).to(dt)
        s["start"], s["len"], s["parent"] = _starts(ql), _rows(kl), _parents(g, ql, 0.0)
        s["max_q"], s["max_kv"], s["scale"] = max(ql), max(kl), 1.0 / math.sqrt(dh)
        reach, live = _reach(s["parent"], s["start"], max(ql))  # the plan is made once a round, for every layer
        s["pos"], s["mask"] = _positions_masks(reach, live, s["start"], s["len"], case["window"])
        s["out"] = torch.zeros((t, nq, dh), dtype=dt, device=DEV)
        s["lse"] = torch.zeros((t, nq), dtype=torch.float32, device=DEV)
    return s


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


def _held(x, exp):
    """What the cache holds of float32 rows [t, n_kv, dh] with an exponent per head, as bf16."""
    e = exp.float()[:, None]
    code, neg, scale = _round4(x * torch.exp2(-e))
    lut = torch.tensor(_E2M1, device=x.device)
    return ((lut[code.int()] * torch.where(neg, -scale, scale)).flatten(-2) * torch.exp2(e)).to(torch.bfloat16)


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


# ------------------------------------------------------------------ trees, plain

def _padded(values, start, n_max, fill):
    """Packed rows as [rows, n_max], and which places are real."""
    i = torch.arange(n_max, device=DEV)
    live = i < (start[1:] - start[:-1])[:, None]
    at = (start[:-1, None] + i).clamp(max=max(values.shape[0] - 1, 0)).long()
    return torch.where(live, values[at], fill) if values.shape[0] else torch.full(live.shape, fill, device=DEV), live


def _reach(parent, start, n_max):
    """reach[r, i, a]: node a of row r is i or one of its ancestors. Paths double in length with each product."""
    par, live = _padded(parent, start, n_max, -1)
    a = torch.arange(n_max, device=DEV)
    reach = ((par[:, :, None] == a) | (a[:, None] == a)).float() * live[:, :, None] * live[:, None, :]
    for _ in range(max(n_max - 1, 1).bit_length()):
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0, live


def _positions_masks(reach, live, start, length, window):
    """Packed positions and four words of mask bits per node."""
    depth = reach.sum(-1) - 1
    base = length - (start[1:] - start[:-1])
    seen = reach & (depth[:, :, None] - depth[:, None, :] < window) if window else reach
    n = live.shape[1]
    bits = torch.nn.functional.pad(seen, (0, MOST - n)).unflatten(-1, (MOST // 32, 32)).long()
    words = (bits << torch.arange(32, device=DEV)).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return (base[:, None] + depth)[live].to(torch.int32), words[live]


# ------------------------------------------------------------------ one pass

def run(state):
    return {"rope": _rope, "prompt": _prompt, "plan": _plan, "tree": _tree, "commit": _commit}[state["case"]["op"]](state)


def _rope(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            b["cache"] = m.kv_q4_cache(s["kc"], s["vc"], s["k_exp"], s["v_exp"])
            b["rope"] = m.mtp_rope(c["rot"], c["theta"])
        m.kv_q4_append_rope(b["cache"], s["q"], s["k"], s["v"], b["rope"], s["pos"], s["slot"], s["q_out"], k_out=s["k_out"], q_norm=s["q_norm"],
                            k_norm=s["k_norm"], eps=EPS)
        m.kv_q4_read(b["cache"], s["slot"], s["k_held"], s["v_held"])
        return {"q": s["q_out"], "k": s["k_out"], "k_held": s["k_held"], "v_held": s["v_held"]}
    half = c["rot"] // 2
    freq = c["theta"] ** (-torch.arange(half, device=DEV, dtype=torch.float64) / max(half, 1))
    angle = s["pos"].double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        x1, x2 = x[..., :half], x[..., half:2 * half]
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., 2 * half:]], -1)

    live = (s["pos"] >= 0)[:, None, None]
    q, k = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"])
    return {"q": torch.where(live, q, 0.0).to(s["q"].dtype), "k": torch.where(live, k, 0.0).to(s["q"].dtype),
            "k_held": torch.where(live, _held(k, s["k_exp"]), 0.0), "v_held": torch.where(live, _held(s["v"].float(), s["v_exp"]), 0.0)}


def _softmax_sum(sc, v, G):
    """Outputs and log sums of scores [..., queries, G, keys] (-inf: out of sight) over values [..., keys, dh]; 0 and -inf where nothing is seen."""
    m_ = sc.amax(-1, keepdim=True)
    m_ = torch.where(m_ == -math.inf, 0.0, m_)
    p = torch.exp(sc.sub_(m_))
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(-3, -2), v).unflatten(-2, (-1, G)) / torch.where(tot > 0, tot, 1.0)
    return o, (m_ + torch.log(tot)).squeeze(-1)


def _prompt(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            b["ws"] = torch.empty(m.kv_attend_prompt_workspace_bytes(s["q"].shape[0], c["rows"]), dtype=torch.uint8, device=DEV)
        m.kv_attend_prompt(s["q"], s["k"], s["v"], s["start"], s["out"], b["ws"], s["max_len"], scale=s["scale"], window=c["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    nq, nkv, L = c["n_q"], c["n_kv"], s["max_len"]
    G, start = nq // nkv, s["start"]
    i = torch.arange(L, device=DEV)
    n = start[1:] - start[:-1]
    at = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()  # [R, L]
    q = s["q"][at].float().unflatten(2, (nkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k, v = (s[x][at].float().transpose(1, 2) for x in ("k", "v"))
    v = torch.where((i < n[:, None])[:, None, :, None], v, 0.0)
    sc = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (L, G)).mul_(s["scale"])
    seen = i <= i[:, None]
    if c["window"]:
        seen &= i > i[:, None] - c["window"]
    sc.masked_fill_(~seen[:, None], -math.inf)
    o, lse = _softmax_sum(sc, v, G)  # [R, nkv, L, G, dh]
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    row = torch.searchsorted(start[1:].contiguous(), t, right=True)
    col = t - start[row]
    return {"out": o[row, :, col].flatten(1, 2).to(s["q"].dtype), "lse": lse[row, :, col].flatten(1, 2)}


def _plan(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        m.kv_tree_plan(s["parent"], s["start"], s["len"], s["pos"], s["mask"], window=c["window"])
        return {"pos": s["pos"], "mask": s["mask"]}
    reach, live = _reach(s["parent"], s["start"], c["n_hi"])
    pos, mask = _positions_masks(reach, live, s["start"], s["len"], c["window"])
    return {"pos": pos, "mask": mask}


def _tree(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            b["cache"] = m.kv_q4_cache(s["kc"], s["vc"], s["k_exp"], s["v_exp"])
            b["ws"] = torch.empty(m.kv_q4_attend_workspace_bytes(b["cache"], c["n_q"], s["max_q"], s["q"].dtype), dtype=torch.uint8, device=DEV)
        m.kv_q4_attend_tree(b["cache"], s["q"], s["table"], s["start"], s["len"], s["mask"], s["out"], b["ws"], s["max_q"], scale=s["scale"],
                            window=c["window"], pos=s["pos"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    nq, nkv, dh, page, R = c["n_q"], c["n_kv"], c["dh"], c["page"], c["rows"]
    G, Q, L = nq // nkv, s["max_q"], s["max_kv"]
    n = s["start"][1:] - s["start"][:-1]
    l = torch.arange(L, device=DEV)
    pages = s["table"][:, l // page].clamp(min=0)

    def cached(cache, exp):  # [R, nkv, L, dh]
        val = _unpack(cache[pages, :, l % page], dh)
        return (val * torch.exp2(exp.float())[:, None]).transpose(1, 2)

    at = (s["start"][:-1, None] + torch.arange(Q, device=DEV)).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][at].float().unflatten(2, (nkv, G)).permute(0, 2, 1, 3, 4).reshape(R, nkv, Q * G, dh)
    sc = torch.matmul(q, cached(s["kc"], s["k_exp"]).transpose(2, 3)).unflatten(2, (Q, G)) * s["scale"]
    node = l - (s["len"] - n)[:, None]  # [R, L]: which node stands at a position; below 0 the common prefix
    word = s["mask"][at].gather(2, (node // 32).clamp(0, MOST // 32 - 1)[:, None].expand(-1, Q, -1).long())
    seen = torch.where((node < 0)[:, None], True, (word >> (node % 32)[:, None]) & 1 > 0) & (node < n[:, None])[:, None]
    if c["window"]:
        seen &= (node >= 0)[:, None] | (l > s["pos"][at][..., None] - c["window"])
    sc.masked_fill_(~seen[:, None, :, None], -math.inf)
    o, lse = _softmax_sum(sc, cached(s["vc"], s["v_exp"]), G)
    t = torch.arange(s["q"].shape[0], device=DEV, dtype=torch.int32)
    row = torch.searchsorted(s["start"][1:].contiguous(), t, right=True)
    col = t - s["start"][row]
    return {"out": o[row, :, col].flatten(1, 2).to(s["q"].dtype), "lse": lse[row, :, col].flatten(1, 2)}


def _commit(s):
    c = s["case"]
    if own:
        import mtp_speculative_decoding_step_gb300 as m
        b = s["buf"]
        if not b:
            b["caches"] = m.kv_q4_caches([m.kv_q4_cache(kv[0], kv[1]) for kv in s["kv"]])
        m.kv_q4_tree_commit(b["caches"], s["table"], s["start"], s["len"], s["parent"], s["tok"], s["choice"], s["n_acc"], s["out_tok"], s["keep"],
                            path=s["path"])
        return {"n_acc": s["n_acc"], "out_tok": s["out_tok"], "keep": s["keep"], "path": s["path"], "kv": s["kv"]}
    N, P, page = c["n_hi"], c["max_path"], c["page"]
    n = s["start"][1:] - s["start"][:-1]
    reach, live = _reach(s["parent"], s["start"], N)
    par, _ = _padded(s["parent"], s["start"], N, -1)
    tok, _ = _padded(s["tok"], s["start"], N, -1)
    choice, _ = _padded(s["choice"], s["start"], N, -1)
    i = torch.arange(N, device=DEV)
    meant = (par >= 0) & live & (tok == choice.gather(1, par.clamp(min=0).long()))
    rival = meant[:, None, :] & (par[:, None, :] == par[:, :, None]) & (i < i[:, None])  # an earlier child of the same node
    good = (meant & ~rival.any(-1)) | ((i == 0) & live)
    on = live & ((reach & ~good[:, None, :]).sum(-1) == 0)  # every node from the root on was chosen
    step = torch.cumsum(on, 1) - 1
    on &= step < P
    n_path = on.sum(1)
    path = torch.full((c["rows"], P + 1), -1, device=DEV, dtype=torch.int64).scatter(1, torch.where(on, step, P), i.expand_as(step))[:, :P]
    after = torch.where(path >= 0, choice.gather(1, path.clamp(min=0)).long(), -1)  # the token behind a node of the path is the next node's, or the target's last
    base = (s["len"] - n).long()
    frm = base[:, None] + path
    to = base[:, None] + torch.arange(P, device=DEV)
    move = path >= 0

    def slot(at):
        return s["table"].long().gather(1, (at // page).clamp(0, s["table"].shape[1] - 1)) * page + at % page

    src, dst = slot(frm)[move], slot(to)[move]
    kv = s["kv"]
    kv[:, :, dst // page, :, dst % page] = kv[:, :, src // page, :, src % page]  # (the right side is read whole first)
    return {"n_acc": (n_path - 1).clamp(min=0).to(torch.int32), "out_tok": after.to(torch.int32), "keep": (base + n_path).to(torch.int32),
            "path": path.to(torch.int32), "kv": kv}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "rope":
        t, dh = case["tokens"], case["dh"]
        values = t * dh * (2 * case["n_q"] + 3 * case["n_kv"])  # q in and out, k in and out, v in
        return {"bytes": values * size + 2 * t * case["n_kv"] * dh * (2 * 9 / 16 + 2) + 12 * t, "flops": 0}  # (+ both caches written, read and given as bf16)
    if op == "prompt":
        n, w = _prompts(case), case["window"] or 1 << 40
        pairs = sum(a * (a + 1) // 2 - max(0, a - w) * (max(0, a - w) + 1) // 2 for a in n)
        return {"bytes": sum(n) * (case["dh"] * 2 * (case["n_q"] + case["n_kv"]) * size + 4 * case["n_q"]), "flops": 4 * case["dh"] * case["n_q"] * pairs}
    if op == "plan":
        return {"bytes": sum(_trees(case)[0]) * (4 + 4 + MOST // 8) + 8 * case["rows"], "flops": 0}
    if op == "commit":
        t = sum(_trees(case)[0])
        return {"bytes": 12 * t + 8 * case["rows"] * (2 + case["max_path"])
                + 2 * 2 * case["layers"] * case["rows"] * min(2, case["max_path"]) * case["n_kv"] * case["dh"] * 9 / 16, "flops": 0}  # (about two rows move)
    slots = pairs = 0
    w = case["window"] or 1 << 40
    for a, b in zip(*_lens(case)):
        slots += min(b, w + a - 1)
        pairs += a * (min(b - a, w - 1) + 1)  # (the prefix, and the node itself)
    q = sum(_lens(case)[0]) * case["n_q"]
    return {"bytes": slots * case["n_kv"] * 2 * case["dh"] * 9 // 16 + q * (2 * case["dh"] * size + 4) + sum(_lens(case)[0]) * MOST // 8,
            "flops": 4 * case["dh"] * case["n_q"] * pairs}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The outputs from the definitions in 64 bits, one row at a time; whole numbers have none."""
    s = prepare(case, seed)
    if case["op"] in ("plan", "commit"):
        return None
    if case["op"] == "rope":
        q, k = _exact_turn(s["q"], s["q_norm"], s["pos"], case), _exact_turn(s["k"], s["k_norm"], s["pos"], case)
        pad = s["pos"] < 0
        out = {"q": q, "k": k, "k_held": _exact_round(k, s["k_exp"]), "v_held": _exact_round(s["v"].double(), s["v_exp"])}
        for x in out.values():
            x[pad] = 0
        return out
    return _exact_prompt(s) if case["op"] == "prompt" else _exact_tree(s)


def _exact_turn(x, w, pos, case):
    x = x.double().clone()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    rot = case["rot"]
    for i in range(rot // 2):  # the pair (i, i + rot / 2) as a complex number, turned
        f = math.exp(-2.0 * i / rot * math.log(case["theta"]))
        z = torch.complex(x[..., i], x[..., i + rot // 2]) * torch.polar(torch.ones_like(pos, dtype=torch.float64), pos.double() * f)[:, None]
        x[..., i], x[..., i + rot // 2] = z.real, z.imag
    return x


def _exact_round(x, exp):
    """The value of {0, .5, 1, 1.5, 2, 3, 4, 6} x block scale nearest to each element; an even code where two are as near."""
    y = x * (2.0 ** -exp.double())[:, None]
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
    return (torch.sign(y) * at * scale).reshape(x.shape) * (2.0 ** exp.double())[:, None]


def _attend64(q, k, v, seen, scale):
    """Out and lse of one head's queries in 64 bits."""
    sc = (q.double() @ k.T) * scale
    sc.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(sc, 1)
    p = torch.exp(sc - lse[:, None])
    p.masked_fill_(~seen, 0.0)
    return p @ v, lse


def _exact_prompt(s):
    c = s["case"]
    G = c["n_q"] // c["n_kv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    start = s["start"].tolist()
    for a, b in zip(start, start[1:]):
        for lo in range(a, b, 2048):  # some queries at a time, and the keys up to the last one's
            hi = min(b, lo + 2048)
            at = torch.arange(lo, hi, device=DEV)[:, None] - torch.arange(a, hi, device=DEV)
            seen = at >= 0
            if c["window"]:
                seen &= at < c["window"]
            for j in range(c["n_q"]):
                out[lo:hi, j], lse[lo:hi, j] = _attend64(s["q"][lo:hi, j], s["k"][a:hi, j // G].double(), s["v"][a:hi, j // G].double(), seen, s["scale"])
    return {"out": out, "lse": lse}


def _exact_tree(s):
    c = s["case"]
    nq, nkv, dh, page = c["n_q"], c["n_kv"], c["dh"], c["page"]
    G = nq // nkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    start, length, parent = s["start"].tolist(), s["len"].tolist(), s["parent"].tolist()
    table = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=DEV)

    def values(cache, row, h, exp):  # [L, dh]
        n = length[row]
        raw = cache[s["table"][row, : -(-n // page)].long(), h].reshape(-1, dh * 9 // 16)[:n]
        byte = raw[:, : dh // 2].long()
        nib = torch.empty((n, dh), dtype=torch.int64, device=DEV)
        nib[:, 0::2], nib[:, 1::2] = byte % 16, byte // 16
        scale = raw[:, dh // 2:].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
        return table[nib % 8] * sign[nib // 8] * scale.repeat_interleave(16, 1) * 2.0 ** int(exp[h])

    for r in range(c["rows"]):
        a, b, n = start[r], start[r + 1], length[r]
        if a == b:
            continue
        prefix = n - (b - a)
        seen = []
        for i in range(b - a):  # up the tree from each node
            up, line = i, []
            while up >= 0:
                line.append(up)
                up = parent[a + up]
            pos = prefix + len(line) - 1
            row = [not c["window"] or p > pos - c["window"] for p in range(prefix)] + [False] * (b - a)
            for back, node in enumerate(line):
                row[prefix + node] = not c["window"] or back < c["window"]
            seen.append(row)
        seen = torch.tensor(seen, device=DEV)
        for h in range(nkv):
            k, v = values(s["kc"], r, h, s["k_exp"]), values(s["vc"], r, h, s["v_exp"])
            for j in range(h * G, h * G + G):
                out[a:b, j], lse[a:b, j] = _attend64(s["q"][a:b, j], k, v, seen, s["scale"])
    return {"out": out, "lse": lse}
