"""Cases and plain forms of the operators that serve many sequences of different lengths from
one pool of cache pages.

  append   rotary encoding of the new rows' k (and q) at their own positions, k and v written to
           their slots of the pages
  prefill  causal grouped-query attention of each sequence's chunk of new rows over its pages,
           optionally with a sliding window and a few first tokens that stay visible (sinks)
  decode   the same for one row per sequence

A sequence of length L with T new rows has them at positions L - T .. L - 1.  Slot p of sequence b
lives in page table[b, p // page], at row p % page of that page.  The row at position p sees slot m
when m <= p and, with a window W > 0, p - W < m or m < sinks.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, **kw):
    c = {"op": op, "dtype": "bf16", "B": 1, "Hq": 24, "Hkv": 8, "d": 128, "page": 64, "ctx_lo": 0, "ctx_hi": 0,
         "q_lo": 1, "q_hi": 1, "window": 0, "sinks": 0, "rope": 0.0, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one generation step of 64 conversations: a new token each, latency alone
        _case("append_step_64", "append", B=64, ctx_lo=0, ctx_hi=32000, rope=1e6, mix=2),
        # a round of prompt chunks of 8 requests, about 16 thousand rows
        _case("append_chunks_8", "append", B=8, ctx_lo=0, ctx_hi=16000, q_lo=600, q_hi=4000, rope=1e6, page=16, mix=3),
        # one short conversation's next token
        _case("decode_one_700", "decode", ctx_lo=699, ctx_hi=699),
        # a serving batch: lengths from a first question to a long document
        _case("decode_batch_32", "decode", B=32, ctx_lo=60, ctx_hi=32000, mix=5),
        # one user's million-token context
        _case("decode_one_1m", "decode", ctx_lo=1048575, ctx_hi=1048575, page=128),
        # window layers of a batch: 1024 newest tokens and four sinks, small pages
        _case("decode_window_64", "decode", B=64, ctx_lo=100, ctx_hi=60000, window=1024, sinks=4, page=16, mix=7),
        # a small fp32 model
        _case("decode_f32_16", "decode", dtype="f32", B=16, Hq=4, Hkv=2, d=64, ctx_lo=100, ctx_hi=8000, mix=8),
        # one fresh prompt
        _case("prefill_first_8192", "prefill", q_lo=8192, q_hi=8192),
        # a mixed round: single tokens, short follow-ups and chunks of longer prompts
        _case("prefill_mixed_12", "prefill", B=12, ctx_lo=10, ctx_hi=16000, q_lo=1, q_hi=500, page=16, mix=10),
        # the next chunk of a long document
        _case("prefill_chunk_512_at_128k", "prefill", ctx_lo=131072, ctx_hi=131072, q_lo=512, q_hi=512, page=128),
        # window layers' prompt chunks, with sinks
        _case("prefill_window_3", "prefill", B=3, ctx_lo=0, ctx_hi=3000, q_lo=1500, q_hi=5000, window=1024, sinks=4, mix=12),
        # a small fp32 model's chunks
        _case("prefill_f32_4", "prefill", dtype="f32", B=4, Hq=4, Hkv=2, d=64, ctx_lo=0, ctx_hi=1500, q_lo=50, q_hi=700,
              page=16, mix=13),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo + 1.0), math.log(hi + 1.0))))) - 1))


def draw(rng):
    op = rng.choice(["append", "prefill", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = 128 if dtype == "bf16" and rng.random() < 0.8 else 64
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if d == 64 or dtype == "f32":
        Hkv, G = min(Hkv, 4), min(G, 4)
    c = _case(None, op, dtype=dtype, d=d, Hkv=Hkv, Hq=Hkv * G, page=rng.choice([16, 32, 64, 128, 256]),
              mix=rng.randrange(1, 1 << 20))
    if op == "append":
        c["B"] = 1 + _log(rng, 0, 63)
        c["ctx_lo"], c["ctx_hi"] = 0, _log(rng, 100, 60000 // c["B"])
        c["q_hi"] = 1 + _log(rng, 0, 12000 // c["B"])
        c["q_lo"] = 1 + _log(rng, 0, c["q_hi"] - 1)
        c["rope"] = rng.choice([0.0, 1e4, 5e6])
    elif op == "decode":
        c["B"] = 1 + _log(rng, 0, 95)
        hi = 4000000 // (c["B"] * Hkv)
        c["ctx_hi"] = _log(rng, 20, hi if dtype == "bf16" else hi // 4)
        c["ctx_lo"] = _log(rng, 0, c["ctx_hi"])
    else:
        c["B"] = 1 + _log(rng, 0, 11)
        # rows and keys together stay below the largest listed product
        c["q_hi"] = 1 + _log(rng, 0, 8000 // c["B"])
        c["q_lo"] = 1 + _log(rng, 0, c["q_hi"] - 1)
        c["ctx_hi"] = _log(rng, 0, min(60000, 1500000000 // (c["B"] * c["q_hi"] * c["Hq"])) if dtype == "bf16" else 3000)
        c["ctx_lo"] = _log(rng, 0, c["ctx_hi"])
    if op != "append" and rng.random() < 0.35:
        c["window"] = 1 + _log(rng, 0, 2000)
        c["sinks"] = rng.choice([0, 1, 4, 100])
    return c


def _lengths(case):
    """(new rows, length with them) of every sequence; they go by the case alone."""
    rng = random.Random(case["mix"])
    T = [1 + _log(rng, case["q_lo"] - 1, case["q_hi"] - 1) for _ in range(case["B"])]
    return T, [_log(rng, case["ctx_lo"], case["ctx_hi"]) + t for t in T]


def prepare(case, seed):
    T, L = _lengths(case)
    B, Hq, Hkv, d, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "page"))
    dt, dev = _DT[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows = sum(T)
    need = [-(-x // page) for x in L]
    pages = sum(need) + 3
    # pages in the order an allocator hands them out after a while: any; unused entries of the table are -1
    order = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((B, max(need)), -1, dtype=np.int32)
    at = np.cumsum([0] + need)
    for b in range(B):
        table[b, :need[b]] = order[at[b]:at[b + 1]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    s = {"case": dict(case), "rows": rows, "max_T": max(T), "scale": d ** -0.5,
         "table": torch.from_numpy(table).to(dev), "lens": torch.tensor(L, dtype=torch.int32, device=dev),
         "cu": torch.tensor(np.cumsum([0] + T), dtype=torch.int32, device=dev),
         "q": normal(rows, Hq, d, std=2.0), "o": torch.empty(rows, Hq, d, dtype=dt, device=dev)}
    if case["op"] == "append":
        s["k_new"], s["v_new"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
        s["k"] = torch.zeros(pages, Hkv, page, d, dtype=dt, device=dev)
        s["v"] = torch.zeros(pages, Hkv, page, d, dtype=dt, device=dev)
    else:
        # page by page in pieces, so that a pool of several GB needs no fp32 copy of itself
        s["k"], s["v"] = (torch.empty(pages, Hkv, page, d, dtype=dt, device=dev).normal_(generator=g) for _ in range(2))
    if own:  # the descriptor and the scratch that a program keeps from call to call
        import gated_retention_shared_gb300 as Y
        s["cache"] = Y.PagedKV(s["k"], s["v"], s["table"], s["lens"], rope_base=case["rope"])
        s["ws"] = torch.empty(Y.yoco_paged_attn_workspace_size(Hq, rows, s["cache"]), dtype=torch.uint8, device=dev)
    return s


def _owner(s):
    """(sequence, row within its chunk, position) of every new row."""
    row = torch.arange(s["rows"], device=s["cu"].device)
    cu, lens = s["cu"].long(), s["lens"].long()
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    t = row - cu[b]
    return b, t, lens[b] - (cu[b + 1] - cu[b]) + t


def _turn(x, pos, base):
    """Rotary encoding: channel pair (2i, 2i+1) of a row at position p turns by p base^(-2i/d)."""
    d = x.shape[-1]
    theta = base ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    angle = torch.remainder(pos.double()[:, None] * theta, 2 * math.pi)
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), -1).reshape(x.shape)


def _append(s):
    b, _, pos = _owner(s)
    base, page = s["case"]["rope"], s["case"]["page"]
    k = _turn(s["k_new"], pos, base).to(s["k"].dtype) if base else s["k_new"]
    q = _turn(s["q"], pos, base).to(s["q"].dtype) if base else s["q"]
    where = s["table"][b, pos // page].long(), pos % page
    s["k"][where[0], :, where[1]] = k
    s["v"][where[0], :, where[1]] = s["v_new"]
    s["o"].copy_(q)
    return s["k"], s["v"], s["o"]


def _pages(s, pos, b):
    """Pages [B, n] that the rows may see a slot of, and the slots' positions [B, n * page] (-1: none)."""
    c, dev = s["case"], pos.device
    B, page, columns = c["B"], c["page"], s["table"].shape[1]
    col = torch.arange(columns, device=dev).expand(B, -1)
    if c["window"]:  # the pages from the first row's window on, and the sinks' pages before them
        first = torch.full((B,), 1 << 40, device=dev).scatter_reduce_(0, b, pos, "amin")
        first = (first - c["window"] + 1).clamp(min=0) // page
        newest = first[:, None] + torch.arange((c["window"] + s["max_T"]) // page + 2, device=dev)
        sink = torch.arange(-(-c["sinks"] // page), device=dev).expand(B, -1)
        col = torch.cat((torch.where(sink < first[:, None], sink, columns), newest), 1)
    there = col < columns
    m = (col[:, :, None] * page + torch.arange(page, device=dev)).masked_fill(~there[:, :, None], -1)
    return s["table"].gather(1, col.clamp(max=columns - 1)).clamp(min=0).long(), m.reshape(B, -1)


def _attention(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    G, T, dev = Hq // Hkv, s["max_T"], s["q"].device
    b, t, pos = _owner(s)
    at = torch.zeros(B, T, dtype=torch.int64, device=dev)
    at[b, t] = pos
    q = torch.zeros(B, T, Hq, d, dtype=torch.float32, device=dev)
    q[b, t] = s["q"].float()
    q = q.reshape(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    table, m = _pages(s, pos, b)
    k = s["k"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).reshape(B, Hkv, T, G, -1)
    del k
    m, p = m[:, None], at[:, :, None]
    seen = (m >= 0) & (m <= p)
    if c["window"]:
        seen &= (m > p - c["window"]) | (m < c["sinks"])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    o = torch.matmul(x.reshape(B, Hkv, T * G, -1), v).reshape(B, Hkv, T, G, d) / total
    o = o.transpose(1, 2).reshape(B, T, Hq, d)
    return o[b, t].to(s["q"].dtype)


def run(s):
    c = s["case"]
    if own:
        import gated_retention_shared_gb300 as Y
        if c["op"] == "append":
            Y.yoco_paged_append(s["k_new"], s["v_new"], s["cache"], s["cu"], q=s["q"], q_out=s["o"], workspace=s["ws"])
            return s["k"], s["v"], s["o"]
        if c["op"] == "decode":
            Y.yoco_paged_attn_decode(s["q"], s["cache"], s["o"], scale=s["scale"], window=c["window"], sinks=c["sinks"],
                                     workspace=s["ws"])
        else:
            Y.yoco_paged_attn_prefill(s["q"], s["cache"], s["cu"], s["o"], scale=s["scale"], window=c["window"],
                                      sinks=c["sinks"], workspace=s["ws"])
        return s["o"]
    if c["op"] == "append":
        return _append(s)
    return _attention(s)


def _seen(p, W, S):
    """How many slots the row at position p sees."""
    if not W or p + 1 <= W:
        return p + 1
    return W + min(S, p + 1 - W)


def _seen_sum(p0, p1, W, S):
    """Sum of _seen over positions p0 .. p1 - 1."""
    def upto(n):  # over 0 .. n - 1
        if not W or n <= W:
            return n * (n + 1) // 2
        full, rest = W * (W + 1) // 2 + (n - W) * W, n - W
        ramp = min(rest, S)
        return full + ramp * (ramp + 1) // 2 + (rest - ramp) * S
    return upto(p1) - upto(p0)


def work(case):
    T, L = _lengths(case)
    Hq, Hkv, d, W, S = (case[k] for k in ("Hq", "Hkv", "d", "window", "sinks"))
    size, rows = (2 if case["dtype"] == "bf16" else 4), sum(T)
    if case["op"] == "append":
        turned = rows * Hq * d * size * 2  # q read and written
        return {"bytes": turned + 2 * 2 * rows * Hkv * d * size, "flops": 3 * rows * (Hq + Hkv) * d if case["rope"] else 0}
    keys = pairs = 0
    for t, n in zip(T, L):
        lo = max(0, n - t - W + 1) if W else 0
        keys += n - lo + min(S if W else 0, lo)
        pairs += _seen_sum(n - t, n, W, S)
    return {"bytes": 2 * rows * Hq * d * size + 2 * keys * Hkv * d * size, "flops": 4 * pairs * Hq * d}


def exact(case, seed):
    """The outputs from the definition in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    T, L = _lengths(case)
    Hq, Hkv, d, page, W, S = (case[k] for k in ("Hq", "Hkv", "d", "page", "window", "sinks"))
    table, first = s["table"].cpu(), np.cumsum([0] + T)
    dev = s["q"].device
    if case["op"] == "append":
        kp, vp, qo = s["k"].double(), s["v"].double(), s["q"].double()
        turn = torch.exp(-torch.arange(0, d, 2, device=dev, dtype=torch.float64) / d * math.log(case["rope"])) if case["rope"] else None
        for b in range(case["B"]):
            p = torch.arange(L[b] - T[b], L[b], device=dev)
            sl = slice(first[b], first[b + 1])
            k, q = s["k_new"][sl].double(), s["q"][sl].double()
            if turn is not None:
                w = torch.polar(torch.ones(len(p), 1, d // 2, device=dev, dtype=torch.float64), (p.double()[:, None] * turn)[:, None])
                k, q = (torch.view_as_real(torch.view_as_complex(z.reshape(*z.shape[:-1], d // 2, 2).contiguous()) * w).reshape(z.shape) for z in (k, q))
            pg = table[b].to(dev).long()[p // page]
            kp[pg, :, p % page], vp[pg, :, p % page], qo[sl] = k, s["v_new"][sl].double(), q
        return kp, vp, qo
    out = torch.empty(s["rows"], Hq, d, dtype=torch.float64, device=dev)
    for b in range(case["B"]):
        ids = table[b, :-(-L[b] // page)].to(dev).long()
        pos = torch.arange(L[b] - T[b], L[b], device=dev)[:, None]
        key = torch.arange(L[b], device=dev)[None]
        hidden = key > pos
        if W:
            hidden |= (key <= pos - W) & (key >= S)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            k = s["k"][ids, hk].reshape(-1, d)[:L[b]].double()
            v = s["v"][ids, hk].reshape(-1, d)[:L[b]].double()
            q = s["q"][first[b]:first[b + 1], h].double()
            a = (q @ k.T * d ** -0.5).masked_fill(hidden, -math.inf)
            a = torch.exp(a - torch.logsumexp(a, 1, keepdim=True))
            out[first[b]:first[b + 1], h] = a @ v
    return out
