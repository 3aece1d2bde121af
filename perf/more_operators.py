"""Cases and plain forms of what a server of models with other scores, positions and page handling
needs next to the paged cache.

  rope      rotary encoding at given positions: pairs (2i, 2i+1) or halves (i, i + r/2) of the first
            r channels, frequencies scaled for long contexts, from strided rows
  append    the same for the new rows' k and q, k and v written to their slots of the pages
  prefill   causal grouped-query attention of chunks of new rows over the pages whose scores are
            capped by a tanh or get a bias by distance, with a prefix mask, a document mask, a window
  decode    the same for one row per sequence
  beam      pages: a round of a search: hypotheses dropped, forked and grown (copy on write)
  churn     pages: a serving round in which sequences end, begin, are cut back and grow
  compact   pages: sequences end, the rest is moved together, others begin

A sequence of length L with T new rows has them at positions L - T .. L - 1.  Slot p of sequence b
lives in page table[b, p // page], at row p % page of that page.  With x = scale q.k the score of the
row at position p for slot m is
    cap tanh(x / cap) - slope_h |p - m|
and the row sees m >= doc_first[row] where (m <= p and (no window, or p - W < m, or m < sinks)) or
m < prefix[b].  A row that sees nothing is zero.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, op, **kw):
    c = {"op": op, "dtype": "bf16", "B": 1, "Hq": 24, "Hkv": 8, "d": 128, "page": 64, "ctx_lo": 0, "ctx_hi": 0,
         "q_lo": 1, "q_hi": 1, "window": 0, "sinks": 0, "cap": 0.0, "bias": False, "prefix": 0, "docs": 0, "tail": 0, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _rope(name, op, **kw):
    c = {"op": op, "dtype": "bf16", "B": 1, "Hq": 24, "Hkv": 8, "d": 128, "page": 64, "ctx_lo": 0, "ctx_hi": 0,
         "q_lo": 1, "q_hi": 1, "rot": 128, "layout": "halves", "scaling": "none", "base": 1e6, "factor": 1.0,
         "original": 8192, "magnitude": 1.0, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _pages_case(name, op, **kw):
    c = {"op": op, "dtype": "bf16", "B": 8, "ways": 0, "Hkv": 8, "d": 128, "page": 64, "len_lo": 100, "len_hi": 1000,
         "grow": 1, "spare": 100, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one generation step of 64 conversations: q and k heads out of a fused projection, latency alone
        _rope("rope_step_64", "rope", q_lo=64, q_hi=64, ctx_hi=60000, rot=128, scaling="by_parts", factor=16.0, magnitude=1.277, mix=2),
        # a round of prompt chunks of 8 requests into the cache, half of each head turned
        _rope("append_chunks_8", "append", B=8, ctx_hi=16000, q_lo=600, q_hi=4000, rot=64, scaling="linear", factor=4.0, page=16, mix=3),
        # one short conversation's next token, scores capped
        _attn("decode_cap_one_700", "decode", ctx_lo=699, ctx_hi=699, cap=50.0),
        # a serving batch of a model with capped scores: from a first question to a long document
        _attn("decode_cap_batch_32", "decode", B=32, ctx_lo=60, ctx_hi=32000, cap=50.0, mix=5),
        # a small fp32 model with a bias by distance, each answer within its own document
        _attn("decode_bias_docs_f32_16", "decode", dtype="f32", B=16, Hq=8, Hkv=2, d=64, ctx_lo=100, ctx_hi=8000, bias=True, docs=1500, mix=8),
        # one fresh prompt of a model with capped scores
        _attn("prefill_cap_4096", "prefill", q_lo=4096, q_hi=4096, cap=30.0),
        # packed documents that do not see one another, and a question at the end that sees them all
        _attn("prefill_docs_8192", "prefill", q_lo=8192, q_hi=8192, docs=700, tail=100),
        # a mixed round of a model with a bias by distance, instructions of each request seen both ways
        _attn("prefill_prefix_bias_12", "prefill", B=12, ctx_lo=10, ctx_hi=12000, q_lo=1, q_hi=500, page=16, bias=True, prefix=600, mix=10),
        # window layers of a small fp32 model with capped scores
        _attn("prefill_cap_f32_4", "prefill", dtype="f32", B=4, Hq=4, Hkv=2, d=64, ctx_hi=1500, q_lo=50, q_hi=700, page=16, cap=20.0,
              window=256, sinks=4, mix=13),
        # a search over 8 requests, three hypotheses more of each
        _pages_case("pages_beam_8x4", "beam", B=8, ways=3, len_lo=200, len_hi=6000, grow=5, mix=14),
        # a serving round of a thousand sequences
        _pages_case("pages_churn_1024", "churn", B=1024, len_lo=20, len_hi=4000, grow=300, page=16, Hkv=2, spare=150000, mix=15),
        # a pool of some GB of which half is moved together, twice
        _pages_case("pages_compact_96", "compact", B=96, len_lo=200, len_hi=16000, mix=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo + 1.0), math.log(hi + 1.0))))) - 1))


def _draw_rope(rng, op):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = _rope(None, op, dtype=dtype, d=d, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), page=rng.choice([16, 32, 64, 128, 256]),
              layout=rng.choice(["pairs", "halves"]), rot=rng.choice([d, d, d // 2, d // 4, 48]), mix=rng.randrange(1, 1 << 20),
              base=rng.choice([1e4, 1e5, 5e6]), scaling=rng.choice(["none", "linear", "ntk", "by_parts"]))
    if c["scaling"] != "none":
        c["factor"], c["magnitude"] = rng.choice([2.0, 8.0, 40.0]), rng.choice([1.0, 1.1])
    c["B"] = 1 if op == "rope" else 1 + _log(rng, 0, 63)
    c["ctx_hi"] = _log(rng, 100, 1000000 if op == "rope" else 60000 // c["B"])
    c["q_hi"] = 1 + _log(rng, 0, 12000 // c["B"])
    c["q_lo"] = 1 + _log(rng, 0, c["q_hi"] - 1)
    return c


def _draw_attn(rng, op):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = 128 if dtype == "bf16" and rng.random() < 0.8 else 64
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if d == 64 or dtype == "f32":
        Hkv, G = min(Hkv, 4), min(G, 4)
    c = _attn(None, op, dtype=dtype, d=d, Hkv=Hkv, Hq=Hkv * G, page=rng.choice([16, 32, 64, 128, 256]), mix=rng.randrange(1, 1 << 20))
    if op == "decode":
        c["B"] = 1 + _log(rng, 0, 63)
        hi = 2500000 // (c["B"] * Hkv)
        c["ctx_hi"] = _log(rng, 20, min(hi, 200000) if dtype == "bf16" else hi // 8)
        c["ctx_lo"] = _log(rng, 0, c["ctx_hi"])
    else:
        c["B"] = 1 + _log(rng, 0, 11)
        c["q_hi"] = 1 + _log(rng, 0, 4000 // c["B"])
        c["q_lo"] = 1 + _log(rng, 0, c["q_hi"] - 1)
        c["ctx_hi"] = _log(rng, 0, min(30000, 400000000 // (c["B"] * c["q_hi"] * c["Hq"])) if dtype == "bf16" else 2000)
        c["ctx_lo"] = _log(rng, 0, c["ctx_hi"])
    while True:
        c["cap"] = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
        c["bias"] = rng.random() < 0.4
        c["docs"] = _log(rng, 20, 3000) if rng.random() < 0.4 else 0
        c["prefix"] = _log(rng, 10, 2000) if rng.random() < 0.4 else 0
        if rng.random() < 0.25:
            c["window"], c["sinks"] = 1 + _log(rng, 0, 2000), rng.choice([0, 1, 4, 100])
        if c["docs"] and rng.random() < 0.5:
            c["tail"] = _log(rng, 1, 100)
        if c["cap"] or c["bias"] or c["docs"] or c["prefix"]:
            return c


def _draw_pages(rng, op):
    c = _pages_case(None, op, dtype=rng.choice(["bf16", "f32"]), Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128, 256]), mix=rng.randrange(1, 1 << 20))
    c["B"] = 2 + _log(rng, 0, 30 if op == "beam" else 700 if op == "churn" else 90)
    c["ways"] = rng.choice([1, 2, 3, 7]) if op == "beam" else 0
    slots = 1200000000 // (2 * c["Hkv"] * c["d"] * (2 if c["dtype"] == "bf16" else 4))  # pools of a GB or so
    c["spare"] = _log(rng, 0, slots // c["page"])
    c["len_hi"] = _log(rng, 50, min(1000000, slots) // (c["B"] * (1 + c["ways"])))
    c["len_lo"] = _log(rng, 0, c["len_hi"])
    c["grow"] = 1 + _log(rng, 0, 300)
    return c


def draw(rng):
    op = rng.choice(["rope", "append", "prefill", "prefill", "decode", "decode", "beam", "churn", "compact"])
    if op in ("rope", "append"):
        return _draw_rope(rng, op)
    if op in ("prefill", "decode"):
        return _draw_attn(rng, op)
    return _draw_pages(rng, op)


# ------------------------------------------------------------------ states

def _lengths(case):
    """(new rows, length with them) of every sequence; they go by the case alone."""
    rng = random.Random(case["mix"])
    T = [1 + _log(rng, case["q_lo"] - 1, case["q_hi"] - 1) for _ in range(case["B"])]
    return T, [_log(rng, case["ctx_lo"], case["ctx_hi"]) + t for t in T]


def _masks(case):
    """(prefix of every sequence, document start of every row); they go by the case alone."""
    T, L = _lengths(case)
    rng = random.Random(case["mix"] + 1)
    prefix = [_log(rng, 0, 2 * case["prefix"]) for _ in L]
    doc = []
    for t, n in zip(T, L):
        starts, at = [], 0
        while at < n and case["docs"]:
            starts.append(at)
            at += 1 + _log(rng, case["docs"] // 4, 2 * case["docs"])
        pos = np.arange(n - t, n)
        first = np.array(starts)[np.searchsorted(starts, pos, side="right") - 1] if starts else np.zeros(t, dtype=np.int64)
        first[pos >= n - case["tail"]] = 0
        doc.append(first)
    return prefix, np.concatenate(doc)


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def _theta(c):
    """Radians per position of the rot / 2 channel pairs."""
    r, f = c["rot"], c["factor"]
    base = c["base"] * f ** (r / (r - 2.0)) if c["scaling"] == "ntk" else c["base"]
    theta = base ** (-2.0 * np.arange(r // 2, dtype=np.float64) / r)
    if c["scaling"] == "linear":
        theta = theta / f
    elif c["scaling"] == "by_parts":  # turns over the original length: from 32 on as they are, up to 1 slowed down
        keep = np.clip((c["original"] * theta / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        theta = theta * (keep + (1.0 - keep) / f)
    return theta


def _table(need, pages, seed, width):
    """A page table of `need` pages for each sequence, in the order that an allocator has after a while."""
    order = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((len(need), width), -1, dtype=np.int32)
    at = np.cumsum([0] + list(need))
    for b, n in enumerate(need):
        table[b, :n] = order[at[b]:at[b + 1]]
    return table


def _pool(case, pages, g):
    shape = (pages, case["Hkv"], case["page"], case["d"])
    return [torch.empty(*shape, dtype=_DT[case["dtype"]], device="cuda").normal_(generator=g) for _ in range(2)]


def _beam_lengths(case):
    rng = random.Random(case["mix"])
    return [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["B"])]


def _page_plan(case):
    """Lengths at the start, and the lengths that the pass's resize calls ask for, in order."""
    n, rng = _beam_lengths(case), random.Random(case["mix"] + 1)
    if case["op"] == "beam":  # parents first, then their children
        start = n + [0] * (case["B"] * case["ways"])
        return start, [start, [x + case["grow"] for x in n * (1 + case["ways"])]]
    if case["op"] == "churn":  # a third ends and begins anew, a third is cut back
        what = [rng.randrange(3) for _ in n]
        low = [0 if w == 0 else max(0, x - case["grow"]) if w == 1 else x for w, x in zip(what, n)]
        return n, [low, [x if w else _log(rng, case["len_lo"], case["len_hi"]) for w, x in zip(what, n)]]
    even = [x if b % 2 else 0 for b, x in enumerate(n)]
    odd = [0 if b % 2 else x for b, x in enumerate(n)]
    return n, [even, n, odd, n]


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, page, d = _DT[case["dtype"]], case["page"], case["d"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    s = {"case": dict(case)}
    if own:
        import gated_retention_shared_gb300 as Y
    if op in ("beam", "churn", "compact"):
        start, asked = _page_plan(case)
        need = [-(-x // page) for x in start]
        most = [max(-(-a[b] // page) for a in [start] + asked) for b in range(len(start))]
        pages = max(sum(need), max(sum(-(-x // page) for x in a) for a in asked)) + len(start) + case["spare"]
        s["k"], s["v"] = _pool(case, pages, g)
        s["table"] = torch.from_numpy(_table(need, pages, seed, max(most) + 1)).to(dev)
        s["lens"], s["asked"] = ints(start), [ints(a) for a in asked]
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        if op == "beam":
            s["src"] = ints(list(range(case["B"])) * case["ways"])
            s["dst"] = ints(range(case["B"], case["B"] * (1 + case["ways"])))
        if own:  # the descriptor and the scratch that a program keeps from call to call
            s["cache"] = Y.PagedKV(s["k"], s["v"], s["table"], s["lens"])
            s["ws"] = torch.empty(Y.yoco_paged_pool_workspace_size(s["cache"]), dtype=torch.uint8, device=dev)
        return s

    T, L = _lengths(case)
    B, Hq, Hkv, rows = case["B"], case["Hq"], case["Hkv"], sum(T)
    s.update(rows=rows, max_T=max(T), lens=ints(L), cu=ints(np.cumsum([0] + T)))
    if op == "rope":
        fused = normal(rows, Hq + 2 * Hkv, d)
        s["x"] = fused[:, :Hq + Hkv]  # q and k of a fused projection
        s["out"] = torch.empty(rows, Hq + Hkv, d, dtype=dt, device=dev)
        first = np.random.RandomState(seed % (1 << 31)).randint(0, case["ctx_hi"] + 1, rows)
        # a step's rows stand anywhere, a chunk's side by side
        s["pos"] = ints(first if rows < 256 else first[0] + np.arange(rows))
    else:
        need = [-(-x // page) for x in L]
        pages = sum(need) + 3
        s["table"] = torch.from_numpy(_table(need, pages, seed, max(need))).to(dev)
        if op == "append":
            s["k_new"], s["v_new"], s["q"] = normal(rows, Hkv, d), normal(rows, Hkv, d), normal(rows, Hq, d)
            s["k"], s["v"] = (torch.zeros(pages, Hkv, page, d, dtype=dt, device=dev) for _ in range(2))
        else:
            s["k"], s["v"] = _pool(case, pages, g)
            s["q"] = normal(rows, Hq, d, std=2.0)
            prefix, doc = _masks(case)
            s["prefix"] = ints(prefix) if case["prefix"] else None
            s["doc"] = ints(doc) if case["docs"] else None
            s["slopes"] = torch.tensor(_slopes(Hq), dtype=torch.float32, device=dev) if case["bias"] else None
            s["scale"] = d ** -0.5
        s["o"] = torch.empty(rows, Hq, d, dtype=dt, device=dev)
    if op in ("rope", "append"):
        if own:
            s["rope"] = Y.Rope(rotary_dim=case["rot"], layout=case["layout"], base=case["base"], scaling=case["scaling"],
                               factor=case["factor"], original=case["original"], low=1.0, high=32.0, magnitude=case["magnitude"])
    elif own:
        s["scores"] = Y.PagedScores(softcap=case["cap"], slopes=s["slopes"], prefix=s["prefix"], doc_first=s["doc"])
    if own and op != "rope":
        s["cache"] = Y.PagedKV(s["k"], s["v"], s["table"], s["lens"])
        s["ws"] = torch.empty(Y.yoco_paged_attn_workspace_size(Hq, rows, s["cache"]), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------- plain forms

def _owner(s):
    """(sequence, row within its chunk, position) of every new row."""
    row = torch.arange(s["rows"], device=s["cu"].device)
    cu, lens = s["cu"].long(), s["lens"].long()
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    t = row - cu[b]
    return b, t, lens[b] - (cu[b + 1] - cu[b]) + t


def _turn(x, pos, c):
    """The first rot channels turned by pos theta and multiplied by the magnitude, the rest as it is."""
    r = c["rot"]
    theta = torch.from_numpy(_theta(c)).to(x.device)
    angle = torch.remainder(pos.double()[:, None] * theta, 2 * math.pi)
    co, si = (torch.cos(angle) * c["magnitude"]).float()[:, None], (torch.sin(angle) * c["magnitude"]).float()[:, None]
    f = x.float()
    if c["layout"] == "pairs":
        x0, x1 = f[..., 0:r:2], f[..., 1:r:2]
        y = torch.stack((x0 * co - x1 * si, x0 * si + x1 * co), -1).flatten(-2)
    else:
        x0, x1 = f[..., :r // 2], f[..., r // 2:r]
        y = torch.cat((x0 * co - x1 * si, x0 * si + x1 * co), -1)
    return torch.cat((y, f[..., r:]), -1).to(x.dtype)


def _append(s):
    b, _, pos = _owner(s)
    page = s["case"]["page"]
    where = s["table"][b, pos // page].long(), pos % page
    s["k"][where[0], :, where[1]] = _turn(s["k_new"], pos, s["case"])
    s["v"][where[0], :, where[1]] = s["v_new"]
    s["o"].copy_(_turn(s["q"], pos, s["case"]))
    return s["k"], s["v"], s["o"]


def _attention(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    G, T, dev = Hq // Hkv, s["max_T"], s["q"].device
    b, t, pos = _owner(s)
    at = torch.full((B, T), -1, dtype=torch.int64, device=dev)
    at[b, t] = pos
    q = torch.zeros(B, T, Hq, d, dtype=torch.float32, device=dev)
    q[b, t] = s["q"].float()
    q = q.reshape(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    table = s["table"].clamp(min=0).long()
    k = s["k"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).reshape(B, Hkv, T, G, -1)
    del k
    if c["cap"]:
        x.div_(c["cap"]).tanh_().mul_(c["cap"])
    m, p, L = torch.arange(x.shape[-1], device=dev), at[:, :, None], s["lens"].long()[:, None, None]
    if c["bias"]:
        x.sub_(s["slopes"].reshape(Hkv, 1, G, 1) * (p - m).abs().float()[:, None, :, None, :])
    seen = m <= p
    if c["window"]:
        seen &= (m > p - c["window"]) | (m < c["sinks"])
    if c["prefix"]:
        seen |= m < s["prefix"].long()[:, None, None]
    seen &= (m < L) & (p >= 0)
    if c["docs"]:
        doc = torch.zeros(B, T, dtype=torch.int64, device=dev)
        doc[b, t] = s["doc"].long()
        seen &= m >= doc[:, :, None]
    seen = seen[:, None, :, None, :]
    x.masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    o = torch.matmul(x.reshape(B, Hkv, T * G, -1), v).reshape(B, Hkv, T, G, d) / torch.where(seen.any(-1, keepdim=True), total, 1.0)
    return o.transpose(1, 2).reshape(B, T, Hq, d)[b, t].to(s["q"].dtype)


def _resize(s, new):
    """The sequences' lengths become `new`: pages behind them go back, pages that are needed are the lowest
    free ones, in the order of the sequences.  A page that is written next and that other sequences have too
    is copied as far as it is filled; where all who have it grow, the first of them keeps it."""
    table, refs, page, dev = s["table"], s["refs"], s["case"]["page"], s["table"].device
    L, N = s["lens"].long(), new.long()
    B, e0, e1 = len(L), (L + page - 1) // page, (N + page - 1) // page
    col = torch.arange(table.shape[1], device=dev)
    drop = (col >= e1[:, None]) & (col < e0[:, None])
    refs -= torch.bincount(table[drop], minlength=len(refs)).to(refs.dtype)
    table[drop] = -1
    seq = torch.arange(B, device=dev)
    held = table[seq, (L // page).clamp(max=table.shape[1] - 1)].clamp(min=0).long()
    grows = (N > L) & (L % page > 0) & (refs[held] > 1)
    owners = torch.bincount(held[grows], minlength=len(refs))
    first = torch.full((len(refs),), B, device=dev).scatter_reduce_(0, held[grows], seq[grows], "amin")
    copied = grows & ~((owners[held] == refs[held]) & (first[held] == seq))
    refs -= torch.bincount(held[copied], minlength=len(refs)).to(refs.dtype)
    need = (e1 - e0).clamp(min=0) + copied
    begin = torch.where(copied, L // page, e0)
    owner = torch.repeat_interleave(seq, need)
    place = torch.arange(len(owner), device=dev) - (need.cumsum(0) - need)[owner]
    pages = (refs == 0).nonzero()[:len(owner), 0]
    table[owner, begin[owner] + place] = pages.to(table.dtype)
    refs[pages] = 1
    src, dst = held[copied], pages[place == 0][copied[owner[place == 0]]]
    filled = (torch.arange(page, device=dev) < (L % page)[copied][:, None])[:, None, :, None]
    s["k"][dst] = torch.where(filled, s["k"][src], s["k"][dst])
    s["v"][dst] = torch.where(filled, s["v"][src], s["v"][dst])
    s["lens"].copy_(new)


def _fork(s):
    """Sequences dst, which are empty, become sequences src on the same pages."""
    src, dst, table = s["src"].long(), s["dst"].long(), s["table"]
    held = (s["lens"].long()[src] + s["case"]["page"] - 1) // s["case"]["page"]
    rows = table[src].masked_fill(torch.arange(table.shape[1], device=table.device) >= held[:, None], -1)
    table[dst] = rows
    s["refs"] += torch.bincount(rows[rows >= 0], minlength=len(s["refs"])).to(s["refs"].dtype)
    s["lens"][dst] = s["lens"][src]


def _compact(s):
    """The pages in use become the first ones: those behind, in order, move to the free ones, in order."""
    refs = s["refs"]
    used = refs > 0
    live = used.sum()
    at = torch.arange(len(refs), device=refs.device)
    src, dst = (used & (at >= live)).nonzero()[:, 0], (~used & (at < live)).nonzero()[:, 0]
    s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    moved = at.clone()
    moved[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, moved[s["table"].clamp(min=0).long()].to(s["table"].dtype), s["table"]))


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import gated_retention_shared_gb300 as Y
        if op == "rope":
            Y.yoco_rope_apply_scaled(s["x"], s["rope"], out=s["out"], positions=s["pos"])
            return s["out"]
        if op == "append":
            Y.yoco_paged_append_rope(s["k_new"], s["v_new"], s["cache"], s["rope"], cu_rows=s["cu"], q=s["q"], q_out=s["o"], workspace=s["ws"])
            return s["k"], s["v"], s["o"]
        if op == "decode":
            Y.yoco_paged_attn_decode_scored(s["q"], s["cache"], s["o"], s["scores"], scale=s["scale"], window=c["window"],
                                            sinks=c["sinks"], workspace=s["ws"])
            return s["o"]
        if op == "prefill":
            Y.yoco_paged_attn_prefill_scored(s["q"], s["cache"], s["cu"], s["o"], s["scores"], scale=s["scale"], window=c["window"],
                                             sinks=c["sinks"], workspace=s["ws"])
            return s["o"]
        Y.yoco_paged_resize(s["cache"], s["refs"], s["asked"][0], workspace=s["ws"])
        if op == "beam":
            Y.yoco_paged_fork(s["cache"], s["refs"], s["src"], s["dst"], workspace=s["ws"])
        elif op == "compact":
            Y.yoco_paged_compact(s["cache"], s["refs"], workspace=s["ws"])
        Y.yoco_paged_resize(s["cache"], s["refs"], s["asked"][1], workspace=s["ws"])
        if op == "compact":
            Y.yoco_paged_resize(s["cache"], s["refs"], s["asked"][2], workspace=s["ws"])
            Y.yoco_paged_compact(s["cache"], s["refs"], workspace=s["ws"])
            Y.yoco_paged_resize(s["cache"], s["refs"], s["asked"][3], workspace=s["ws"])
        return s["table"], s["lens"], s["refs"], s["k"], s["v"]
    if op == "rope":
        s["out"].copy_(_turn(s["x"], s["pos"], c))
        return s["out"]
    if op == "append":
        return _append(s)
    if op in ("prefill", "decode"):
        return _attention(s)
    _resize(s, s["asked"][0])
    if op == "beam":
        _fork(s)
    elif op == "compact":
        _compact(s)
    _resize(s, s["asked"][1])
    if op == "compact":
        _resize(s, s["asked"][2])
        _compact(s)
        _resize(s, s["asked"][3])
    return s["table"], s["lens"], s["refs"], s["k"], s["v"]


# -------------------------------------------------------------------- work

def work(case):
    size, op, d = (2 if case["dtype"] == "bf16" else 4), case["op"], case["d"]
    if op in ("beam", "churn", "compact"):
        start, asked = _page_plan(case)
        page, at, held, moved = case["page"], start, [-(-x // case["page"]) for x in start], 0
        entries = 0
        slot = 2 * 2 * case["Hkv"] * d * size  # k and v read and written
        for a in asked:
            now = [-(-x // page) for x in a]
            entries += sum(abs(x - y) for x, y in zip(held, now))
            if op == "compact" and sum(a) < sum(start):  # those that stay lie behind those that end, from the second pass on
                moved += min(sum(now), sum(start_pages(case)) - sum(now)) * page * slot
            at, held = a, now
        if op == "beam":  # each child but the parent copies what its last page holds
            moved = case["ways"] * sum(x % page for x in start) * slot
            entries += case["ways"] * sum(-(-x // page) for x in start) * 2
        return {"bytes": moved + 8 * entries + 12 * len(start) * len(asked), "flops": 0}
    T, L = _lengths(case)
    Hq, Hkv, rows = case["Hq"], case["Hkv"], sum(T)
    if op == "rope":
        return {"bytes": 2 * rows * (Hq + Hkv) * d * size + 4 * rows, "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    if op == "append":
        return {"bytes": 2 * rows * (Hq + 2 * Hkv) * d * size, "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    keys = pairs = 0
    for lo, pre, hi in _spans(case):
        # the slots that some row of the sequence sees, and those that its rows see in all
        keys += _union(lo, pre, hi)
        pairs += int((hi - lo).sum() + (np.minimum(pre[:, 1], lo) - np.minimum(pre[:, 0], lo)).sum() +
                     (np.maximum(pre[:, 1], hi) - np.maximum(pre[:, 0], hi)).sum())
    return {"bytes": 2 * rows * Hq * d * size + 2 * keys * Hkv * d * size, "flops": 4 * pairs * Hq * d}


def start_pages(case):
    return [-(-x // case["page"]) for x in _page_plan(case)[0]]


def _spans(case):
    """Of every sequence, for its rows: the run [lo, hi) of slots up to the row, and the run `pre` of prefix or sinks."""
    T, L = _lengths(case)
    prefix, doc = _masks(case)
    first = 0
    for b, (t, n) in enumerate(zip(T, L)):
        pos, dc = np.arange(n - t, n), doc[first:first + t] if case["docs"] else np.zeros(t, dtype=np.int64)
        first += t
        hi = pos + 1
        lo = np.minimum(np.maximum(dc, hi - case["window"] if case["window"] else 0), hi)
        head = np.minimum(case["sinks"], hi) if case["window"] else np.zeros(t, dtype=np.int64)
        head = np.maximum(head, min(prefix[b], n) if case["prefix"] else 0)
        yield lo, np.stack((np.minimum(dc, head), head), 1), hi


def _union(lo, pre, hi):
    n = int(max(hi.max(), pre.max()))
    mark = np.zeros(n + 1, dtype=np.int64)
    for a, b in ((lo, hi), (pre[:, 0], pre[:, 1])):
        np.add.at(mark, a, 1)
        np.add.at(mark, b, -1)
    return int((np.cumsum(mark)[:n] > 0).sum())


# ------------------------------------------------------------------- exact

def _exact_turn(x, pos, c):
    r = c["rot"]
    half = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    lnb = math.log(c["base"]) + (math.log(c["factor"]) * r / (r - 2.0) if c["scaling"] == "ntk" else 0.0)
    w = torch.exp(-2.0 * half / r * lnb)
    if c["scaling"] == "linear":
        w = w / c["factor"]
    if c["scaling"] == "by_parts":
        turns = c["original"] * w / (2 * math.pi)
        part = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        w = part * w + (1.0 - part) * w / c["factor"]
    z = torch.polar(torch.full((len(pos), 1, r // 2), c["magnitude"], device=x.device, dtype=torch.float64), (pos.double()[:, None] * w)[:, None])
    y = x.double().clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if c["layout"] == "pairs" else (slice(0, r // 2), slice(r // 2, r))
    u = torch.complex(y[..., a], y[..., b]) * z
    y[..., a], y[..., b] = u.real, u.imag
    return y


def exact(case, seed):
    """The outputs from the definition in 64 bits, sequence by sequence; of the page operators the pools alone, in whole pages."""
    op, page = case["op"], case["page"]
    s = prepare(case, seed)
    if op == "rope":
        return _exact_turn(s["x"], s["pos"].long(), case)
    if op in ("beam", "churn", "compact"):
        return _exact_pages(s, case)
    T, L = _lengths(case)
    table, first, dev = s["table"].cpu(), np.cumsum([0] + T), s["q"].device
    if op == "append":
        kp, vp, qo = s["k"].double(), s["v"].double(), s["q"].double()
        for b in range(case["B"]):
            p = torch.arange(L[b] - T[b], L[b], device=dev)
            sl = slice(first[b], first[b + 1])
            pg = table[b].to(dev).long()[p // page]
            kp[pg, :, p % page] = _exact_turn(s["k_new"][sl], p, case)
            vp[pg, :, p % page] = s["v_new"][sl].double()
            qo[sl] = _exact_turn(s["q"][sl], p, case)
        return kp, vp, qo
    Hq, Hkv, W, S = (case[k] for k in ("Hq", "Hkv", "window", "sinks"))
    prefix, doc = _masks(case)
    slopes = _slopes(Hq)
    out = torch.zeros(s["rows"], Hq, case["d"], dtype=torch.float64, device=dev)
    for b in range(case["B"]):
        ids = table[b, :-(-L[b] // page)].to(dev).long()
        pos = torch.arange(L[b] - T[b], L[b], device=dev)[:, None]
        key = torch.arange(L[b], device=dev)[None]
        hidden = key > pos
        if W:
            hidden |= (key <= pos - W) & (key >= S)
        if case["prefix"]:
            hidden &= key >= prefix[b]
        if case["docs"]:
            hidden |= key < torch.from_numpy(doc[first[b]:first[b + 1]]).to(dev)[:, None]
        empty = hidden.all(1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            k = s["k"][ids, hk].reshape(-1, case["d"])[:L[b]].double()
            v = s["v"][ids, hk].reshape(-1, case["d"])[:L[b]].double()
            a = s["q"][first[b]:first[b + 1], h].double() @ k.T * case["d"] ** -0.5
            if case["cap"]:
                a = case["cap"] * torch.tanh(a / case["cap"])
            if case["bias"]:
                a = a - float(np.float32(slopes[h])) * (key - pos).abs()
            a = a.masked_fill(hidden, -math.inf)
            a = torch.exp(a - torch.logsumexp(a, 1, keepdim=True)) @ v
            out[first[b]:first[b + 1], h] = a.masked_fill(empty[:, None], 0.0)
    return out


def _exact_pages(s, case):
    """A pass sequence by sequence and page by page, on the host; page contents as (page at the start, slots of it) pieces."""
    page = case["page"]
    table = [[int(x) for x in row if x >= 0] for row in s["table"].cpu().numpy()]
    lens = [int(x) for x in s["lens"].cpu()]
    count = [int(x) for x in s["refs"].cpu()]
    P = len(count)
    source = np.tile(np.arange(P)[:, None], (1, page))  # page at the start that each slot's contents come from

    def resize(new):
        for b, n in enumerate(new):
            keep = -(-n // page)
            for p in table[b][keep:]:
                count[p] -= 1
            del table[b][keep:]
        growing = [b for b, n in enumerate(new) if n > lens[b]]
        tails = [(b, table[b][-1]) for b in growing if lens[b] % page and count[table[b][-1]] > 1]
        have = {}
        for b, p in tails:
            have.setdefault(p, []).append(b)
        copies = {b: p for b, p in tails if not (len(have[p]) == count[p] and have[p][0] == b)}
        for p in copies.values():
            count[p] -= 1
        free = iter([p for p in range(P) if count[p] == 0])
        for b in growing:
            if b in copies:
                p = next(free)
                count[p] = 1
                source[p, :lens[b] % page] = source[copies[b], :lens[b] % page]
                table[b][-1] = p
            while len(table[b]) < -(-new[b] // page):
                p = next(free)
                count[p] = 1
                table[b].append(p)
        lens[:] = new

    def fork():
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            table[b], lens[b] = list(table[a]), lens[a]
            for p in table[a]:
                count[p] += 1

    def compact():
        live = sum(n > 0 for n in count)
        to = dict(zip([p for p in range(live, P) if count[p]], [p for p in range(live) if not count[p]]))
        for a, b in to.items():
            source[b] = source[a]
            count[a], count[b] = 0, count[a]
        for row in table:
            row[:] = [to.get(p, p) for p in row]

    asked = _page_plan(case)[1]
    resize(asked[0])
    if case["op"] == "beam":
        fork()
    if case["op"] == "compact":
        compact()
    resize(asked[1])
    if case["op"] == "compact":
        resize(asked[2])
        compact()
        resize(asked[3])
    at = torch.from_numpy(source).to(s["k"].device)
    slot = torch.arange(page, device=at.device)[None].expand(P, -1)
    changed = (at != torch.arange(P, device=at.device)[:, None]).any(1)
    out = []
    for x in (s["k"], s["v"]):
        y = x.clone()
        y[changed] = x.transpose(1, 2)[at[changed], slot[changed]].transpose(1, 2)
        out.append(y)
    return [None, None, None] + out
