"""GPU checks of the scored paged calls: capped scores, biases by distance, prefix and document
masks, against the definition in 64 bits, element by element.

The bounds are those of the plain calls (tests/test_gpu_paged.py: a score is off by (d + 2) u S,
each weight by that and a few u, the sums by n u, all twice for numerator and denominator, weights
rounded to bf16 for the tensor cores by 2^-8 at most) with, for what comes after q.k, with Y the
largest |cap tanh(x / cap)| and B the largest slope * distance of the slots that the row sees,
  cap    eta Y: eta = 1.5e-6 on the tensor cores (a polynomial of relative error 1.01e-6 or
         exponential and reciprocal of 2^-22 each, and six roundings), else 16 u (a polynomial of 6e-8
         or exponential and reciprocal of 4 u and 2 u, of which at most 0.76 come through, and as many).  (It does not enlarge the error of its argument: its slope is at most 1.)
  bias   8 u (Y + B): the slope times log2(e), the product, and the sum, in two steps
each twice as well.  On the tensor cores run bf16 at head size 128 and its prefills at 64, by one kernel:
o = sum(round(p) v) / sum(p), in which |round(p) - p| <= 2^-8 p (half a step of bf16), so o is off by at most
2^-8 sum(p |v|) / sum(p) for it, as for the plain calls at 128.
"""
import math

import numpy as np
import pytest
import torch

import test_gpu_paged as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)]


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32)


def reference(pool, Q, b, pos, doc, prefix, cap, slopes, window, sinks, scale, decode=False):
    T, Hq, d = Q.shape
    bf16 = Q.dtype == torch.bfloat16
    tensor = bf16 and (d == 128 or not decode)
    L = pool.lens[b]
    out, tol = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    m, p = torch.arange(L)[None], pos[:, None]
    seen = m <= p
    if window:
        seen &= (m > p - window) | (m < sinks)
    seen = (seen | (m < prefix)) & (m >= doc[:, None]) & (p >= 0)
    none = ~seen.any(1)
    far = (m - p).abs().double()
    for h in range(Hq):
        k, v = pool.rows(b, h // (Hq // pool.Hkv))
        k, v = torch.nan_to_num(k), torch.nan_to_num(v)
        x = Q[:, h].double() @ k.T * scale
        if cap:
            x = cap * torch.tanh(x / cap)
        top = x.abs().masked_fill(~seen, 0).amax(1, keepdim=True)
        B = torch.zeros_like(top)
        if slopes is not None:
            bias = float(slopes[h]) * far
            x, B = x - bias, bias.abs().masked_fill(~seen, 0).amax(1, keepdim=True)
        w = torch.softmax(x.masked_fill(~seen, -math.inf), 1).masked_fill(none[:, None], 0.0)
        o = w @ v
        S = (Q[:, h].double().abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(1, keepdim=True)
        e = U * (2 * (d + 4) * S + 2 * seen.sum(1, keepdim=True) + 16)
        e = e + (2 * (1.5e-6 if tensor else 16 * U) * top if cap else 0) + (16 * U * (top + B) if slopes is not None else 0)
        rounded, half = (2.0 ** -8 if tensor else 0.0, 2.0 ** -8) if bf16 else (0.0, U)
        out[:, h], tol[:, h] = o, half * o.abs() + (e + rounded) * (w @ v.abs()) + 1e-30
    return out, tol


def check(got, pool, Q, cu, doc, prefix, cap, slopes, window, sinks, scale, decode=False):
    got = got.cpu().double()
    for b in range(len(pool.lens)):
        T = cu[b + 1] - cu[b]
        if T == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(T) + pool.lens[b] - T
        ref, tol = reference(pool, Q[rows].cpu(), b, pos, doc[rows], prefix[b], cap, slopes, window, sinks, scale, decode)
        off = (got[rows] - ref).abs()
        assert torch.isfinite(off).all(), (b, "not finite", int((~torch.isfinite(off)).sum()))
        worst = float((off / tol).max())
        assert worst <= 1.0, (b, worst, float(off.max()))


def documents(lens, new, size, seed, tail=0):
    """The document starts of each sequence's new rows; the last `tail` see everything."""
    g = np.random.RandomState(seed)
    rows = []
    for n, t in zip(lens, new):
        starts = [0]
        while starts[-1] < n:
            starts.append(starts[-1] + 1 + g.randint(2 * size))
        pos = np.arange(n - t, n)
        first = np.array(starts)[np.maximum(np.searchsorted(starts, pos, side="right") - 1, 0)]
        first[max(0, t - tail):] = 0 if tail else first[max(0, t - tail):]
        rows.append(first)
    return torch.from_numpy(np.concatenate(rows) if rows else np.zeros(0)).long()


def cuda_ints(x):
    return torch.as_tensor(x).to(torch.int32).cuda()


def run(Y, new, ctx, Hq, Hkv, d, page, dtype, cap=0.0, bias=False, prefix=None, docs=0, tail=0, doc=None, window=0, sinks=0,
        std=2.0, seed=5, decode=False, slopes=None):
    lens = [t + c for t, c in zip(new, ctx)]
    pool = P.Pool(Y, lens, Hkv, d, page, dtype, seed=seed)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    g = torch.Generator().manual_seed(seed + 100)
    extra = 0 if decode else 3
    Q = (torch.randn(cu[-1] + extra, Hq, d, generator=g) * std).to(P.DT[dtype]).cuda()
    O = torch.full_like(Q, 7.0)
    if doc is None and docs:
        doc = documents(lens, new, docs, seed, tail)
    rows_doc = torch.zeros(cu[-1], dtype=torch.int64) if doc is None else doc
    sl = slopes if slopes is not None else slopes_of(Hq) if bias else None
    scores = Y.PagedScores(cap, None if sl is None else sl.cuda(), None if prefix is None else cuda_ints(prefix),
                           None if doc is None else cuda_ints(torch.cat((doc, torch.zeros(extra, dtype=torch.int64)))))
    ws = torch.full((Y.yoco_paged_attn_workspace_size(Hq, Q.shape[0], pool.dev),), 0xA5, dtype=torch.uint8, device="cuda")
    if decode:
        Y.yoco_paged_attn_decode_scored(Q, pool.dev, O, scores, window=window, sinks=sinks, workspace=ws)
    else:
        Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cuda_ints(cu), O, scores, window=window, sinks=sinks, workspace=ws)
    Y.yoco_workspace_status(ws)
    check(O, pool, Q, cu, rows_doc.clamp(min=0), [0] * len(lens) if prefix is None else prefix, cap, sl, window, sinks, d ** -0.5, decode)
    assert bool((O[cu[-1]:] == 7.0).all())  # rows behind the last sequence
    return pool, Q, O, scores


FORMS = {
    "cap": dict(cap=30.0),
    "low cap": dict(cap=1.5),  # most scores outside the polynomial's range
    "high cap": dict(cap=4e5),  # a cap that changes nothing must cost nothing
    "bias": dict(bias=True),
    "cap bias": dict(cap=8.0, bias=True),
    "docs": dict(docs=60),
    "docs tail": dict(docs=150, tail=20),
    "prefix": dict(prefix="some"),
    "prefix bias": dict(prefix="some", bias=True),
    "all": dict(cap=20.0, bias=True, prefix="some", docs=90, tail=5),
    "window cap": dict(cap=20.0, window=100, sinks=4),
    "window bias docs": dict(bias=True, window=200, sinks=30, docs=200),
    "window prefix bias": dict(bias=True, prefix="some", window=37, sinks=2),
    "window all": dict(cap=10.0, bias=True, prefix="some", docs=120, tail=9, window=64, sinks=100),
}


def form(name, lens):
    f = dict(FORMS[name])
    if f.get("prefix") == "some":
        f["prefix"] = [(37 * (b + 1) * 7) % (n + 20) for b, n in enumerate(lens)]
    return f


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("dtype,d", TYPES)
def test_decode(Y, dtype, d, name):
    ctx = [0, 6, 127, 128, 700, 1500, 15, 300]
    run(Y, [1] * 8, ctx, 6, 2, d, 16, dtype, decode=True, **form(name, [c + 1 for c in ctx]))


@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 64), (4, 4, 128), (10, 2, 32), (16, 1, 1024), (32, 2, 256)])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_decode_heads_and_pages(Y, dtype, d, Hq, Hkv, page):
    run(Y, [1] * 4, [3000, 50, 9, 800], Hq, Hkv, d, page, dtype, decode=True, cap=25.0, bias=True, docs=400)


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("dtype,d", TYPES)
def test_prefill(Y, dtype, d, name):
    new, ctx = [1, 0, 70, 200, 300, 5, 129], [0, 9, 500, 3, 40, 1000, 0]
    run(Y, new, ctx, 6, 2, d, 16, dtype, **form(name, [a + b for a, b in zip(new, ctx)]))


@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 64), (4, 4, 128), (10, 2, 32), (16, 1, 1024), (32, 2, 256)])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_prefill_heads_and_pages(Y, dtype, d, Hq, Hkv, page):
    run(Y, [90, 33, 1], [400, 0, 2000], Hq, Hkv, d, page, dtype, cap=25.0, bias=True, docs=150, prefix=[200, 20, 0], tail=3)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("name", ["cap", "docs tail", "prefix bias", "window all"])
def test_prefill_cut_into_pieces(Y, dtype, d, name):
    """Few rows over many keys: the keys are cut and joined, with rows that see nothing of a piece."""
    new, ctx = [5, 40], [9000, 3000]
    f = form(name, [9005, 3040])
    if "docs" in f:
        f["docs"] = 2500
    run(Y, new, ctx, 6, 2, d, 64, dtype, **f)


def test_prefix_longer_than_the_rows(Y):
    """A whole prompt that sees itself both ways, and prefixes past the end and below zero."""
    for dtype, d in TYPES:
        run(Y, [300, 200, 64, 10], [0, 0, 100, 0], 6, 2, d, 16, dtype, prefix=[300, 1 << 30, -5, 4], bias=True)
        run(Y, [300, 200], [0, 500], 6, 2, d, 16, dtype, prefix=[250, 600], window=50, sinks=2, bias=True, cap=10.0)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_rows_that_see_nothing_are_zero(Y, dtype, d):
    """Documents that start behind their rows (padding), some rows or whole row blocks, and whole sequences."""
    new = [200, 50, 30]
    doc = torch.zeros(280, dtype=torch.int64)
    doc[60:] = 1 << 29
    doc[150:200] = 40
    doc[200:230] = 2147483647
    doc[230:250] = -7
    for pre in (None, [0, 20, 0]):
        _, _, O, _ = run(Y, new, [100, 0, 7], 6, 2, d, 16, dtype, doc=doc, prefix=pre)
        assert bool((O[250:280] == 0).all()) and bool((O[60:150] == 0).all())
    _, _, O, _ = run(Y, [1] * 3, [100, 0, 7], 6, 2, d, 16, dtype, doc=torch.tensor([101, 1, 3]), decode=True)
    assert bool((O[:2] == 0).all())


@pytest.mark.parametrize("dtype,d", TYPES)
def test_slots_before_every_document_may_hold_anything(Y, dtype, d):
    """Pages that no row sees are NaN, given back or named by no entry at all."""
    lens, page = [700, 300], 16
    pool = P.Pool(Y, lens, 2, d, page, dtype)
    g = torch.Generator().manual_seed(3)
    for decode in (False, True):
        new = [1, 1] if decode else [60, 40]
        first = [500, 100]
        k, v, table = pool.k.clone(), pool.v.clone(), pool.table.clone()
        for b in range(2):
            p = torch.arange(first[b])
            k[pool.table[b].long()[p // page], :, p % page] = math.nan
            v[pool.table[b].long()[p // page], :, p % page] = math.nan
            table[b, :first[b] // page] = -1
        cache = Y.PagedKV(k.cuda(), v.cuda(), table.cuda(), cuda_ints(lens))
        doc = torch.cat([torch.full((t,), f) for t, f in zip(new, first)])
        doc[0] += 0 if decode else 30
        Q = (torch.randn(sum(new), 6, d, generator=g) * 2).to(P.DT[dtype]).cuda()
        O = torch.empty_like(Q)
        ws = torch.zeros(Y.yoco_paged_attn_workspace_size(6, Q.shape[0], cache), dtype=torch.uint8, device="cuda")
        s = Y.PagedScores(doc_first=cuda_ints(doc))
        if decode:
            Y.yoco_paged_attn_decode_scored(Q, cache, O, s, workspace=ws)
        else:
            Y.yoco_paged_attn_prefill_scored(Q, cache, cuda_ints([0, 60, 100]), O, s, workspace=ws)
        Y.yoco_workspace_status(ws)
        cu = [0] + list(np.cumsum(new))
        check(O, pool, Q, [int(x) for x in cu], doc, [0, 0], 0.0, None, 0, 0, d ** -0.5)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_infinite_and_nan_scores(Y, dtype, d):
    """A cap makes infinite scores finite, on both sides; a NaN key poisons the rows that see it, and those only."""
    lens, new = [300], [200]
    pool = P.Pool(Y, lens, 1, d, 16, dtype)
    big = 3e38 if dtype == "f32" else 3.3e38

    def put(p, value):
        pool.k[pool.table[0].long()[p // 16], 0, p % 16] = value
    put(10, big)
    put(30, -big)
    cache = Y.PagedKV(pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), cuda_ints(lens))
    Q = torch.full((200, 2, d), 2.0, dtype=P.DT[dtype], device="cuda")
    O = torch.empty_like(Q)
    s = Y.PagedScores(softcap=5.0)
    Y.yoco_paged_attn_prefill_scored(Q, cache, cuda_ints([0, 200]), O, s)
    k, v = pool.rows(0, 0)
    x = (2.0 * k.sum(1) * d ** -0.5).clamp(-1e300, 1e300)
    x = 5.0 * torch.tanh(x / 5.0)
    for r in (0, 100, 199):
        w = torch.softmax(x[:101 + r], 0)
        # all q equal: a score is off by (d + 2) u |x|, far below a weight's rounding
        assert torch.allclose(O[r, 0].cpu().double(), w @ v[:101 + r], rtol=0, atol=(2.0 ** -6 if dtype == "bf16" else 1e-4))
    put(150, math.nan)
    cache = Y.PagedKV(pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), cuda_ints(lens))
    Y.yoco_paged_attn_prefill_scored(Q, cache, cuda_ints([0, 200]), O, s)
    bad = torch.isnan(O).any(-1).any(-1).cpu()
    assert bool(bad[50:].all()) and not bool(bad[:50].any())  # row r is at position 100 + r
    One = torch.empty(1, 2, d, dtype=P.DT[dtype], device="cuda")
    Y.yoco_paged_attn_decode_scored(Q[:1], cache, One, s)
    assert bool(torch.isnan(One).all())
    Y.yoco_paged_attn_decode_scored(Q[:1], cache, One, Y.PagedScores(softcap=5.0, doc_first=cuda_ints([151])))
    assert bool(torch.isfinite(One).all())


@pytest.mark.parametrize("dtype,d", TYPES)
def test_slopes_of_any_sign_and_none(Y, dtype, d):
    sl = torch.tensor([0.0, -0.02, 0.5, 3.0, 1e-4, 0.0])
    run(Y, [150, 1], [60, 900], 6, 2, d, 16, dtype, slopes=sl, prefix=[170, 0])
    run(Y, [1, 1], [260, 900], 6, 2, d, 16, dtype, slopes=sl, decode=True)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_nothing_set_gives_the_plain_calls_bits(Y, dtype, d):
    pool, Q, O, s = run(Y, [130, 7], [700, 90], 6, 2, d, 16, dtype, window=300, sinks=4)
    o = torch.full_like(O, 7.0)
    Y.yoco_paged_attn_prefill(Q, pool.dev, cuda_ints([0, 130, 137]), o, window=300, sinks=4)
    assert torch.equal(O, o)
    pool, Q, O, s = run(Y, [1, 1, 1], [700, 0, 90], 6, 2, d, 16, dtype, decode=True)
    o = torch.empty_like(O)
    Y.yoco_paged_attn_decode(Q, pool.dev, o)
    assert torch.equal(O, o)


def test_calls_captured_into_a_graph_follow_the_device_values(Y):
    new, ctx = [40, 80], [300, 20]
    lens = [340, 100]
    pool = P.Pool(Y, lens, 2, 128, 16, "bf16")
    cu = cuda_ints([0, 40, 120])
    g = torch.Generator().manual_seed(1)
    Q = (torch.randn(120, 6, 128, generator=g) * 2).to(torch.bfloat16).cuda()
    O = torch.zeros_like(Q)
    prefix, doc, slopes = cuda_ints([0, 0]), cuda_ints([0] * 120), slopes_of(6).cuda()
    s = Y.PagedScores(15.0, slopes, prefix, doc)
    ws = torch.empty(Y.yoco_paged_attn_workspace_size(6, 120, pool.dev), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cu, O, s, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cu, O, s, workspace=ws)
    for pre, first in (([0, 0], 0), ([200, 50], 0), ([10, 100], 60)):
        prefix.copy_(cuda_ints(pre))
        doc.fill_(first)
        graph.replay()
        torch.cuda.synchronize()
        check(O, pool, Q, [0, 40, 120], torch.full((120,), first), pre, 15.0, slopes_of(6), 0, 0, 128 ** -0.5)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("cap", [3.0, 7.0, 12.0, 19.99, 20.0, 60.0])
def test_caps_about_the_size_of_the_products(Y, cap, dtype, d, decode):
    """Products on both sides of the polynomials' ends, with and without a bias."""
    new, ctx = ([1, 1, 1], [400, 0, 900]) if decode else ([70, 1, 130], [300, 20, 0])
    for bias in (False, True):
        run(Y, new, ctx, 6, 2, d, 16, dtype, cap=cap, bias=bias, decode=decode)


@pytest.mark.parametrize("std", [0.5, 3.0, 8.0])
@pytest.mark.parametrize("cap", [19.99, 20.0, 44.99, 45.0, 100.0])
def test_products_about_the_ends_of_the_polynomials(Y, cap, std):
    """Each degree's neighbours, with products from within its range to past it; masked and whole tiles."""
    for bias in (False, True):
        run(Y, [130, 40], [300, 0], 6, 2, 128, 16, "bf16", cap=cap, bias=bias, std=std, docs=170)
    run(Y, [1, 1, 1], [300, 0, 900], 6, 2, 128, 16, "bf16", cap=cap, std=std, decode=True)


def test_same_bits_every_time(Y):
    pool, Q, O, s = run(Y, [200, 300, 5], [3000, 3, 6000], 6, 2, 128, 16, "bf16", cap=20.0, bias=True, docs=500, prefix=[50, 200, 9])
    first = O.clone()
    for _ in range(3):
        Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cuda_ints([0, 200, 500, 505]), O, s)
        assert torch.equal(O, first)


@pytest.mark.parametrize("B", [33, 300])
def test_many_sequences(Y, B):
    g = np.random.RandomState(B)
    new, ctx = [int(x) for x in g.randint(0, 40, B)], [int(x) for x in g.randint(0, 400, B)]
    run(Y, new, ctx, 4, 2, 128, 16, "bf16", cap=20.0, docs=100, prefix=[int(x) for x in g.randint(0, 100, B)])
    run(Y, [1] * B, ctx, 4, 2, 128, 16, "bf16", cap=20.0, docs=100, decode=True)


def test_more_row_blocks_than_are_planned_one_by_one(Y):
    """4096 sequences with documents: planned by sequences, as they would be by row blocks."""
    g = np.random.RandomState(7)
    new, ctx = [int(x) for x in g.randint(0, 3, 4096)], [int(x) for x in g.randint(0, 60, 4096)]
    run(Y, new, ctx, 1, 1, 64, 16, "f32", docs=20)


def test_overlapping_row_bounds_with_documents(Y):
    """Bounds that fall back give two sequences the same rows: all of them are planned and written."""
    pool = P.Pool(Y, [1000] * 5, 1, 64, 16, "f32")
    Q = torch.randn(1000, 1, 64, device="cuda")
    O = torch.full_like(Q, 7.0)
    s = Y.PagedScores(doc_first=cuda_ints([0] * 1000))
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(1, 1000, pool.dev), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cuda_ints([0, 1000, 0, 1000, 0, 1000]), O, s, workspace=ws)
    with pytest.raises(Y.YocoError) as e:
        Y.yoco_workspace_status(ws)
    assert e.value.status == Y.YOCO_ERR_INVALID_ARG
    pos = torch.arange(1000)
    refs = [reference(pool, Q.cpu(), b, pos, torch.zeros(1000, dtype=torch.int64), 0, 0.0, None, 0, 0, 0.125) for b in (0, 2, 4)]
    # blocks of the three sequences write the same rows, a few channels to a thread, in any order
    ok = torch.stack([(O.cpu().double() - r).abs() <= t for r, t in refs]).any(0)
    assert bool(ok.all())


def test_bad_metadata_is_recorded_and_reads_nothing_outside(Y):
    """Row bounds that decrease and lengths past the table: recorded, the sound sequences' rows are right."""
    pool = P.Pool(Y, [100, 80], 2, 128, 16, "bf16")
    Q = torch.randn(60, 4, 128, device="cuda").to(torch.bfloat16)
    O = torch.zeros_like(Q)
    doc = cuda_ints([0] * 60)
    s = Y.PagedScores(10.0, None, cuda_ints([5, 5]), doc)
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(4, 60, pool.dev), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_prefill_scored(Q, pool.dev, cuda_ints([0, 60, 30]), O, s, workspace=ws)
    with pytest.raises(Y.YocoError) as e:
        Y.yoco_workspace_status(ws)
    assert e.value.status == Y.YOCO_ERR_INVALID_ARG
    check(O[:60], pool, Q[:60], [0, 60, 60], torch.zeros(60, dtype=torch.int64), [5, 5], 10.0, None, 0, 0, 128 ** -0.5)
