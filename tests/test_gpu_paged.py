"""GPU checks of the paged cache: appends, chunk and single-token attention, windows with
sinks, against the definition in 64 bits.

Every pool starts as NaN, so a slot that the definition does not read (past a sequence's
length, in a page of another sequence, in a page that the window has left) poisons the
result if a kernel lets it in.

Bounds, element by element, with A = sum_m softmax_m |v_m| and S = scale sum_c |q_c k_c| at
its largest over the row's slots, u = 2^-24, n slots, d channels:
  a score is a sum of d products in fp32, off by at most (d + 2) u S; each weight is then
  off by that factor and a few u for the exponential and its argument (|x| log2 e u <= 2 S u),
  and the two sums by n u:     e32 = u (2 (d + 4) S + 2 n + 16)
  |o - o64| <= h |o64| + (e32 + w) A + tiny, h half a step of the output's type (2^-8 for
  bf16, 2^-24 for fp32), w = 2^-8 where the weights are rounded to bf16 for the tensor cores
  and 0 otherwise (the bound with 2^-8 is used for every bf16 case at head size 128).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


class Pool:
    """Random pages for sequences of the given lengths; everything they do not hold is NaN."""

    def __init__(self, Y, lens, Hkv, d, page, dtype, seed=1, spare=2, room=0, rope=0.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.Hkv, self.d = list(lens), page, Hkv, d
        need = [-(-(n + room) // page) for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.k = torch.full((pages, Hkv, page, d), math.nan, dtype=DT[dtype])
        self.v = self.k.clone()
        for b, n in enumerate(lens):
            p = torch.arange(n)
            ids = self.table[b].long()[p // page]
            self.k[ids, :, p % page] = torch.randn(n, Hkv, d, generator=g).to(DT[dtype])
            self.v[ids, :, p % page] = torch.randn(n, Hkv, d, generator=g).to(DT[dtype])
        self.dev = Y.PagedKV(self.k.cuda(), self.v.cuda(), self.table.cuda(),
                             torch.tensor(self.lens, dtype=torch.int32).cuda(), rope_base=rope)

    def rows(self, b, hk):
        p = torch.arange(self.lens[b])
        ids = self.table[b].long()[p // self.page]
        return self.k[ids, hk, p % self.page].double(), self.v[ids, hk, p % self.page].double()


def reference(pool, Q, b, pos, scale, window, sinks):
    """(o, bound) in 64 bits of rows Q [T, Hq, d] of sequence b at positions pos."""
    T, Hq, d = Q.shape
    bf16 = Q.dtype == torch.bfloat16
    out, tol = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    m = torch.arange(pool.lens[b])[None]
    seen = m <= pos[:, None]
    if window:
        seen &= (m > pos[:, None] - window) | (m < sinks)
    none = ~seen.any(1)
    for h in range(Hq):
        k, v = pool.rows(b, h // (Hq // pool.Hkv))
        k, v = torch.nan_to_num(k), torch.nan_to_num(v)
        q = Q[:, h].double()
        x = (q @ k.T * scale).masked_fill(~seen, -math.inf)
        p = torch.softmax(x, 1).masked_fill(none[:, None], 0.0)
        o = p @ v
        S = (q.abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(1, keepdim=True) if seen.shape[1] else torch.zeros(T, 1)
        e32 = U * (2 * (d + 4) * S + 2 * seen.sum(1, keepdim=True) + 16)
        w, half = (2.0 ** -8 if d == 128 else 0.0, 2.0 ** -8) if bf16 else (0.0, U)
        out[:, h], tol[:, h] = o, half * o.abs() + (e32 + w) * (p @ v.abs()) + 1e-30
    return out, tol


def check(got, pool, Q, cu, scale, window, sinks):
    got = got.cpu().double()
    for b in range(len(pool.lens)):
        T = cu[b + 1] - cu[b]
        if T == 0:
            continue
        q = Q[cu[b]:cu[b + 1]].cpu()
        pos = torch.arange(T) + pool.lens[b] - T
        ref, tol = reference(pool, q, b, pos, scale, window, sinks)
        off = (got[cu[b]:cu[b + 1]] - ref).abs()
        assert torch.isfinite(off).all(), (b, "not finite", int((~torch.isfinite(off)).sum()))
        worst = float((off / tol).max())
        assert worst <= 1.0, (b, worst, float(off.max()))


def run_decode(Y, lens, Hq, Hkv, d, page, dtype, window=0, sinks=0, seed=3, std=2.0):
    pool = Pool(Y, lens, Hkv, d, page, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed + 100)
    Q = (torch.randn(len(lens), Hq, d, generator=g) * std).to(DT[dtype]).cuda()
    O = torch.full_like(Q, math.nan)
    ws = torch.full((Y.yoco_paged_attn_workspace_size(Hq, len(lens), pool.dev),), 0xA5, dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_decode(Q, pool.dev, O, window=window, sinks=sinks, workspace=ws)
    Y.yoco_workspace_status(ws)
    check(O, pool, Q, list(range(len(lens) + 1)), d ** -0.5, window, sinks)
    return pool, Q, O


def run_prefill(Y, new, ctx, Hq, Hkv, d, page, dtype, window=0, sinks=0, seed=5, std=2.0, tail=3):
    lens = [t + c for t, c in zip(new, ctx)]
    pool = Pool(Y, lens, Hkv, d, page, dtype, seed=seed)
    cu = [0] + list(np.cumsum(new))
    g = torch.Generator().manual_seed(seed + 100)
    Q = (torch.randn(cu[-1] + tail, Hq, d, generator=g) * std).to(DT[dtype]).cuda()
    O = torch.full_like(Q, 7.0)
    ws = torch.full((Y.yoco_paged_attn_workspace_size(Hq, Q.shape[0], pool.dev),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    Y.yoco_paged_attn_prefill(Q, pool.dev, torch.tensor(cu, dtype=torch.int32, device="cuda"), O, window=window,
                              sinks=sinks, workspace=ws)
    Y.yoco_workspace_status(ws)
    check(O, pool, Q, [int(x) for x in cu], d ** -0.5, window, sinks)
    assert bool((O[cu[-1]:] == 7.0).all())  # rows behind the last sequence
    return pool, Q, O


# ------------------------------------------------------------------ append

def turned(x, pos, base):
    d = x.shape[-1]
    if not base:
        return x.double()
    a = pos.double()[:, None] * torch.tensor(base, dtype=torch.float64) ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    x = x.double()
    y = torch.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return y


def close_turn(got, x, pos, base, dtype):
    """One rounding to the type, and the angle: its fixed-point form is off by below 2^-31 turns, its
    float form by 2^-25 of half a turn, sine and cosine by 2^-23: together below 2^-20 of the pair's size."""
    ref = turned(x, pos, base)
    size = torch.sqrt(x.double()[..., 0::2] ** 2 + x.double()[..., 1::2] ** 2).repeat_interleave(2, -1)
    half = 2.0 ** -8 if dtype == "bf16" else U
    bound = half * ref.abs() + (2.0 ** -20 * size if base else 0.0)
    assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() - bound).max())


def strided(x, how):
    """x [rows, heads, d] on the GPU as a view with other strides."""
    rows, heads, d = x.shape
    if how == "dense":
        return x.cuda()
    if how == "fused":  # a part of a wider row
        big = torch.zeros(rows, heads + 3, d, dtype=x.dtype, device="cuda")
        big[:, 1:1 + heads] = x.cuda()
        return big[:, 1:1 + heads]
    big = torch.zeros(heads, rows + 5, d, dtype=x.dtype, device="cuda")  # head-major staging
    big[:, :rows] = x.cuda().transpose(0, 1)
    return big[:, :rows].transpose(0, 1)


@pytest.mark.parametrize("new,ctx,Hq,Hkv,d,page,dtype,rope,how", [
    ([1, 1, 1], [0, 5, 700], 6, 2, 128, 64, "bf16", 1e6, "dense"),
    ([5, 0, 130, 1], [0, 9, 61, 16], 3, 3, 64, 16, "bf16", 1e4, "fused"),
    ([70, 3], [1000000, 16383], 4, 1, 128, 128, "bf16", 5e6, "heads"),
    ([33, 2, 0], [7, 0, 0], 4, 2, 64, 32, "f32", 1e4, "heads"),
    ([17], [100], 16, 1, 128, 16, "f32", 0.0, "fused"),
    ([400, 300, 500], [0, 10, 20], 24, 8, 128, 256, "bf16", 0.0, "dense"),
])
def test_append(Y, new, ctx, Hq, Hkv, d, page, dtype, rope, how):
    lens = [a + b for a, b in zip(new, ctx)]
    if max(lens) > 100000:  # a far position: pages only where rows are written
        pool = Pool(Y, [0] * len(lens), Hkv, d, page, dtype, spare=6, rope=rope)
        table = torch.full((len(lens), -(-max(lens) // page)), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(lens):
            for e in range((n - new[b]) // page, -(-n // page)):
                table[b, e], at = at, at + 1
        pool.table = table
        pool.dev = Y.PagedKV(pool.k.cuda(), pool.v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             rope_base=rope)
    else:
        pool = Pool(Y, lens, Hkv, d, page, dtype, rope=rope)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    rows = cu[-1] + 2  # two rows behind the last sequence
    g = torch.Generator().manual_seed(11)
    k, v, q = (torch.randn(rows, h, d, generator=g).to(DT[dtype]) for h in (Hkv, Hkv, Hq))
    q_out = torch.full((rows, Hq, d), 9.0, dtype=DT[dtype], device="cuda")
    before_k, before_v = pool.dev.k.cpu(), pool.dev.v.cpu()
    cu_d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws = torch.full((256,), 0xA5, dtype=torch.uint8, device="cuda")
    Y.yoco_paged_append(strided(k, how), strided(v, how), pool.dev, cu_d, q=strided(q, how), q_out=q_out, workspace=ws)
    Y.yoco_workspace_status(ws)
    after_k, after_v, q_got = pool.dev.k.cpu(), pool.dev.v.cpu(), q_out.cpu()
    assert bool((q_got[cu[-1]:] == 9.0).all())
    for b, T in enumerate(new):
        pos = torch.arange(T) + ctx[b]
        ids = pool.table[b].long()[pos // page]
        sl = slice(cu[b], cu[b + 1])
        close_turn(after_k[ids, :, pos % page], k[sl], pos, rope, dtype)
        close_turn(q_got[sl], q[sl], pos, rope, dtype)
        assert torch.equal(after_v[ids, :, pos % page], v[sl])
        if not rope:
            assert torch.equal(after_k[ids, :, pos % page], k[sl]) and torch.equal(q_got[sl], q[sl])
        before_k[ids, :, pos % page] = after_k[ids, :, pos % page]
        before_v[ids, :, pos % page] = after_v[ids, :, pos % page]
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(before_k.view(bits), after_k.view(bits))  # every other slot as it was
    assert torch.equal(before_v.view(bits), after_v.view(bits))


def test_append_one_row_each_q_in_place_and_q_alone(Y):
    lens = [1, 17, 64, 300]
    pool = Pool(Y, lens, 2, 128, 16, "bf16", rope=1e4)
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(4, h, 128, generator=g).bfloat16() for h in (2, 2, 6))
    pos = torch.tensor(lens) - 1
    qd = q.cuda()
    Y.yoco_paged_append(k.cuda(), v.cuda(), pool.dev, q=qd)
    close_turn(qd.cpu(), q, pos, 1e4, "bf16")
    kk = pool.dev.k.cpu()
    for b in range(4):
        p = int(pos[b])
        close_turn(kk[pool.table[b, p // 16], :, p % 16][None], k[b:b + 1], pos[b:b + 1], 1e4, "bf16")
    q2, before = q.cuda(), pool.dev.k.clone()
    out = torch.empty_like(q2)
    Y.yoco_paged_append(None, None, pool.dev, q=q2, q_out=out)
    assert torch.equal(out, qd) and torch.equal(q2.cpu(), q)
    assert torch.equal(before.view(torch.int16), pool.dev.k.view(torch.int16))


# ------------------------------------------------------------------ decode

def test_calls_of_no_rows_do_nothing(Y):
    pool = Pool(Y, [7, 0], 2, 128, 16, "bf16")
    before = pool.dev.k.clone()
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y.yoco_paged_append(kv, kv, pool.dev, cu, q=none)
    Y.yoco_paged_attn_prefill(none, pool.dev, cu, torch.empty_like(none))
    assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(pool.dev.k))


def test_append_of_one_row_and_one_head_with_any_stride_on_those_axes(Y):
    pool = Pool(Y, [7], 1, 128, 16, "bf16", rope=1e4)
    k, v, q = (torch.randn(1, h, 128).bfloat16() for h in (1, 1, 4))
    odd = [torch.as_strided(x.cuda(), x.shape, (3, 128 if x.shape[1] > 1 else 5, 1)) for x in (k, v, q)]
    Y.yoco_paged_append(odd[0], odd[1], pool.dev, q=odd[2])
    page = int(pool.table[0, 0])
    pos = torch.tensor([6])
    close_turn(pool.dev.k.cpu()[page, :, 6][None], k, pos, 1e4, "bf16")
    close_turn(odd[2].cpu(), q, pos, 1e4, "bf16")
    assert torch.equal(pool.dev.v.cpu()[page, :, 6][None], v)


TYPES = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)]


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 3), (1, 16), (3, 2), (2, 5), (1, 9)])
def test_decode_lengths_from_none_to_many(Y, dtype, d, Hkv, G):
    run_decode(Y, [0, 1, 2, 16, 17, 127, 128, 129, 1000, 0, 2500], Hkv * G, Hkv, d, 16, dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (128, 130), (700, 1), (5000, 3)])
def test_decode_pages_windows_and_sinks(Y, page, window, sinks):
    run_decode(Y, [1, 130, 131, 900, 3000], 6, 2, 128, page, "bf16", window, sinks)


@pytest.mark.parametrize("dtype,d", TYPES[1:])
@pytest.mark.parametrize("window,sinks", [(1, 1), (200, 0), (200, 300)])
def test_decode_window_types(Y, dtype, d, window, sinks):
    run_decode(Y, [1, 130, 600, 2000], 4, 2, d, 32, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_one_long_sequence_is_split_and_joined(Y, dtype):
    run_decode(Y, [60001], 4, 2, 128, 64, dtype)


def test_decode_many_short_sequences(Y):
    lens = [(37 * i * i + 5) % 301 for i in range(700)]
    run_decode(Y, lens, 3, 1, 128, 16, "bf16")


@pytest.mark.parametrize("dtype,d", TYPES)
def test_decode_peaked_and_growing_scores(Y, dtype, d):
    """Large scores: the running maximum moves all the time and most weights vanish."""
    run_decode(Y, [50, 700, 3000], 6, 2, d, 64, dtype, std=12.0)


def test_decode_ignores_pages_left_behind_by_the_window(Y):
    """Pages wholly out of sight may be given back: their table entries name nothing."""
    pool, Q, O = run_decode(Y, [2000, 900], 4, 2, 128, 32, "bf16", 100, 5)
    pool.dev.page_table[0, 1:(2000 - 100) // 32] = 1 << 30
    O2 = torch.full_like(O, math.nan)
    ws = torch.empty(Y.yoco_paged_attn_workspace_size(4, 2, pool.dev), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_decode(Q, pool.dev, O2, window=100, sinks=5, workspace=ws)
    Y.yoco_workspace_status(ws)
    assert torch.equal(O, O2)


# ----------------------------------------------------------------- prefill

@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 3), (1, 16), (1, 7)])
def test_prefill_ragged(Y, dtype, d, Hkv, G):
    run_prefill(Y, [1, 0, 2, 43, 130, 300], [0, 5, 700, 100, 0, 33], Hkv * G, Hkv, d, 16, dtype)


@pytest.mark.parametrize("page", [16, 64, 128, 512])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 4), (128, 130), (300, 1)])
def test_prefill_pages_windows_and_sinks(Y, page, window, sinks):
    run_prefill(Y, [1, 200, 513], [1000, 900, 77], 6, 2, 128, page, "bf16", window, sinks)


@pytest.mark.parametrize("dtype,d", TYPES[1:])
@pytest.mark.parametrize("window,sinks", [(1, 1), (90, 0), (90, 200)])
def test_prefill_window_types(Y, dtype, d, window, sinks):
    run_prefill(Y, [3, 150], [700, 260], 4, 2, d, 32, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 64, 90])
def test_prefill_few_rows_long_context_is_split_and_joined(Y, dtype, T):
    run_prefill(Y, [T], [20000], 6, 2, 128, 64, dtype)


def test_prefill_many_rows(Y):
    run_prefill(Y, [2100], [0], 6, 2, 128, 64, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_one_long_sequence_among_many_short_ones(Y, dtype):
    run_prefill(Y, [30] * 40 + [100], [50] * 40 + [9000], 8, 8, 128, 64, dtype)


@pytest.mark.parametrize("B", [2, 16, 31, 32, 33, 256, 257])
def test_prefill_of_as_many_sequences_as_a_way_of_planning_takes(Y, B):
    new = [(5 * b + 2) % 9 for b in range(B - 1)] + [90]
    run_prefill(Y, new, [(31 * b) % 200 for b in range(B - 1)] + [5000], 2, 1, 128, 16, "bf16")


def test_prefill_of_hundreds_of_sequences_and_a_long_one(Y):
    run_prefill(Y, [2, 0, 1] * 100 + [70, 3], [3, 40, 0] * 100 + [6000, 900], 2, 1, 128, 16, "bf16")


@pytest.mark.parametrize("dtype,d", TYPES)
def test_prefill_peaked_scores(Y, dtype, d):
    run_prefill(Y, [300, 20], [200, 1500], 6, 2, d, 64, dtype, std=12.0)


def test_prefill_of_more_sequences_than_a_warp_looks_up_at_once(Y):
    new = [(7 * i) % 5 for i in range(150)]
    run_prefill(Y, new, [(31 * i) % 90 for i in range(150)], 2, 1, 128, 16, "bf16")


# ------------------------------------------------------- bad lengths and pages

def status(Y, ws):
    try:
        Y.yoco_workspace_status(ws)
    except Y.YocoError as e:
        return e.status
    return 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_the_table_cannot_hold_count_as_empty(Y, dtype):
    pool = Pool(Y, [100, 50, 70], 2, 128, 16, dtype)
    Q = torch.randn(3, 4, 128).to(DT[dtype]).cuda()
    O = torch.full_like(Q, math.nan)
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(4, 3, pool.dev), dtype=torch.uint8, device="cuda")
    for bad in (-1, 100000, -2 ** 31, 2 ** 31 - 1):
        pool.dev.seq_lens[1] = bad
        Y.yoco_paged_attn_decode(Q, pool.dev, O, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG
        assert bool((O[1] == 0).all()) and bool(torch.isfinite(O.float()).all())
        O.fill_(math.nan)
        Y.yoco_paged_attn_prefill(Q, pool.dev, torch.arange(4, dtype=torch.int32, device="cuda"), O, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG
        assert bool((O[1] == 0).all()) and bool(torch.isfinite(O.float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_outside_the_pool_are_reported_and_not_touched(Y, dtype):
    pool = Pool(Y, [100, 50], 2, 128, 16, dtype)
    Q = torch.randn(2, 4, 128).to(DT[dtype]).cuda()
    O = torch.empty_like(Q)
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(4, 2, pool.dev), dtype=torch.uint8, device="cuda")
    cu = torch.arange(3, dtype=torch.int32, device="cuda")
    for bad in (-1, pool.dev.c.num_pages, 2 ** 31 - 1):
        pool.dev.page_table[0, 6] = bad  # the page of slots 96 .. 99
        Y.yoco_paged_attn_decode(Q, pool.dev, O, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG and bool(torch.isfinite(O.float()).all())
        Y.yoco_paged_attn_prefill(Q, pool.dev, cu, O, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG and bool(torch.isfinite(O.float()).all())
        before = pool.dev.k.clone()
        kv = torch.ones(2, 2, 128, dtype=DT[dtype], device="cuda")
        Y.yoco_paged_append(kv, kv, pool.dev, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG
        pg, row = int(pool.table[1, 3]), 49 % 16
        before[pg, :, row] = 1.0  # sequence 1 is written all the same
        assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(pool.dev.k))


def test_bad_row_bounds_are_reported(Y):
    pool = Pool(Y, [100, 50, 60], 2, 128, 16, "bf16")
    Q = torch.randn(12, 4, 128).bfloat16().cuda()
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(4, 12, pool.dev), dtype=torch.uint8, device="cuda")
    for cu in ([0, 5, 3, 12], [0, 4, 8, 13], [-2, 4, 8, 12], [0, 2 ** 31 - 1, 8, 12]):
        O = torch.full_like(Q, 7.0)
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        Y.yoco_paged_attn_prefill(Q, pool.dev, cud, O, workspace=ws)
        assert status(Y, ws) == Y.YOCO_ERR_INVALID_ARG
        assert bool(torch.isfinite(O.float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_overlapping_row_bounds_stay_within_the_work_list(Y, dtype):
    """cu_rows that fall back to 0 count the call's rows many times over, more row blocks than
    the list of work has room for; what follows the output and the workspace stays as it was."""
    B, rows = 64, 640
    pool = Pool(Y, [2500] * 2 + [700] * (B - 2), 1, 128, 64, dtype)
    Q = torch.randn(rows, 4, 128).to(DT[dtype]).cuda()
    n = Y.yoco_paged_attn_workspace_size(4, rows, pool.dev)
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    ws[n:] = 0x5A
    O = torch.full((rows + 8, 4, 128), 7.0, dtype=DT[dtype], device="cuda")
    cu = torch.tensor([0, rows] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    Y.yoco_paged_attn_prefill(Q, pool.dev, cu, O[:rows], workspace=ws[:n])
    assert status(Y, ws[:n]) == Y.YOCO_ERR_INVALID_ARG
    assert bool(torch.isfinite(O.float()).all()) and bool((O[rows:] == 7.0).all()) and bool((ws[n:] == 0x5A).all())


def test_more_new_rows_than_the_sequence_holds(Y):
    """Rows at negative positions see nothing: zeros from attention, left out by the append."""
    pool = Pool(Y, [10, 100], 2, 128, 16, "bf16", rope=1e4)
    cu = torch.tensor([0, 25, 27], dtype=torch.int32, device="cuda")
    Q = torch.randn(27, 4, 128).bfloat16().cuda()
    O = torch.full_like(Q, math.nan)
    Y.yoco_paged_attn_prefill(Q, pool.dev, cu, O)
    assert bool((O[:15] == 0).all())
    got = O.cpu().double()
    ref, tol = reference(pool, Q[15:25].cpu(), 0, torch.arange(10), 128 ** -0.5, 0, 0)
    assert bool(((got[15:25] - ref).abs() <= tol).all())
    out = torch.full_like(Q, 5.0)
    kv = torch.randn(27, 2, 128).bfloat16().cuda()
    Y.yoco_paged_append(kv, kv, pool.dev, cu, q=Q, q_out=out)
    assert bool((out[:15] == 5.0).all()) and not bool((out[15:] == 5.0).any())
    assert torch.equal(pool.dev.v[int(pool.table[0, 0]), :, :10].transpose(0, 1), kv[15:25])


# ------------------------------------------------------------- large extents

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_pools_past_32_bits_of_elements(Y, dtype, d):
    """The sequence's pages lie behind 2^31 elements of each tensor (2^32 bytes and more)."""
    pool = Pool(Y, [300, 77], 2, d, 64, dtype)
    lead = (2 ** 31) // (2 * 64 * d)
    n = lead + pool.k.shape[0]
    big = [torch.empty(n, 2, 64, d, dtype=DT[dtype], device="cuda") for _ in range(2)]
    for t, small in zip(big, (pool.k, pool.v)):
        t[:2] = math.nan
        t[lead:] = small.cuda()
    table = torch.where(pool.table >= 0, pool.table + lead, pool.table)
    dev = Y.PagedKV(big[0], big[1], table.cuda(), pool.dev.seq_lens)
    Q = torch.randn(2, 6, d, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    O = torch.empty_like(Q)
    Y.yoco_paged_attn_decode(Q, dev, O)
    check(O, pool, Q, [0, 1, 2], d ** -0.5, 0, 0)
    O.fill_(math.nan)
    Y.yoco_paged_attn_prefill(Q, dev, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), O)
    check(O, pool, Q, [0, 1, 2], d ** -0.5, 0, 0)
    kv = torch.randn(2, 2, d).to(DT[dtype]).cuda()
    Y.yoco_paged_append(kv, kv, dev)
    for b, L in enumerate(pool.lens):
        assert torch.equal(big[0][int(table[b, (L - 1) // 64]), :, (L - 1) % 64], kv[b])
    assert bool(big[0][:2].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_as_many_sequences_as_a_call_takes(Y, dtype):
    lens = [(7 * b) % 40 for b in range(4096)]
    run_decode(Y, lens, 1, 1, 128, 16, dtype)
    new = [min(n, b % 3) for b, n in enumerate(lens)]
    run_prefill(Y, new, [n - t for n, t in zip(lens, new)], 1, 1, 128, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(15000, 100), (9000, 0), (300, 12000)])
def test_long_windows_and_many_sinks_are_split_and_joined(Y, dtype, window, sinks):
    run_prefill(Y, [5, 1], [20000, 100], 2, 1, 128, 64, dtype, window=window, sinks=sinks)
    run_decode(Y, [20000, 100], 2, 1, 128, 64, dtype, window=window, sinks=sinks)


# ----------------------------------------------------------- used together

def serve(Y, pool, steps, k, v, q, window, sinks):
    """Feed every sequence's rows in the given chunks: append, then attend; outputs per sequence."""
    B, d = len(pool.lens), pool.d
    done, outs = [0] * B, [[] for _ in range(B)]
    for new in steps:
        cu = [0] + [int(x) for x in np.cumsum(new)]
        rows = [torch.arange(done[b], done[b] + new[b]) for b in range(B)]
        take = lambda x: torch.cat([x[b][rows[b]] for b in range(B)]).cuda()  # noqa: E731
        done = [a + n for a, n in zip(done, new)]
        pool.dev.seq_lens.copy_(torch.tensor(done, dtype=torch.int32))
        kk, vv, qq = take(k), take(v), take(q)
        if new == [1] * B:
            Y.yoco_paged_append(kk, vv, pool.dev, q=qq)
            o = torch.empty_like(qq)
            Y.yoco_paged_attn_decode(qq, pool.dev, o, window=window, sinks=sinks)
        else:
            cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
            Y.yoco_paged_append(kk, vv, pool.dev, cud, q=qq)
            o = torch.empty_like(qq)
            Y.yoco_paged_attn_prefill(qq, pool.dev, cud, o, window=window, sinks=sinks)
        for b in range(B):
            outs[b].append(o[cu[b]:cu[b + 1]].cpu())
    return [torch.cat(x) for x in outs]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_chunks_then_tokens_equal_the_whole_sequence(Y, dtype, d, window, sinks):
    Hq, Hkv, page, base = 6, 2, 16, 1e4
    steps = [[100, 0, 7], [33, 260, 1], [1, 1, 1], [1, 1, 1], [0, 40, 2], [1, 1, 1]]
    total = [sum(s[b] for s in steps) for b in range(3)]
    pool = Pool(Y, total, Hkv, d, page, dtype, rope=base)
    pool.dev.k.fill_(math.nan)
    pool.dev.v.fill_(math.nan)
    g = torch.Generator().manual_seed(9)
    k, v, q = ([torch.randn(n, h, d, generator=g).to(DT[dtype]) * s for n in total] for h, s in ((Hkv, 1), (Hkv, 1), (Hq, 2)))
    outs = serve(Y, pool, steps, k, v, q, window, sinks)
    pool.k, pool.v = pool.dev.k.cpu(), pool.dev.v.cpu()  # the keys as stored (turned, rounded)
    for b in range(3):
        pos = torch.arange(total[b])
        kk = torch.stack([pool.rows(b, h)[0] for h in range(Hkv)], 1)
        close_turn(kk, k[b], pos, base, dtype)
        # the turned query as stored: from the q-only append
        pool.dev.seq_lens.copy_(torch.tensor(total, dtype=torch.int32))
        qq = torch.cat(q).cuda()
        cu = torch.tensor([0] + list(np.cumsum(total)), dtype=torch.int32, device="cuda")
        Y.yoco_paged_append(None, None, pool.dev, cu, q=qq)
        sl = slice(sum(total[:b]), sum(total[:b + 1]))
        ref, tol = reference(pool, qq[sl].cpu(), b, pos, d ** -0.5, window, sinks)
        assert bool(((outs[b].double() - ref).abs() <= tol).all())


def test_shared_prefix_pages(Y):
    """Two sequences that name the same pages for their common prefix."""
    pool = Pool(Y, [320, 320], 2, 128, 64, "bf16")
    pool.table[1, :4] = pool.table[0, :4]
    pool.dev.page_table.copy_(pool.table)
    Q = torch.randn(2, 4, 128).bfloat16().cuda()
    O = torch.empty_like(Q)
    Y.yoco_paged_attn_decode(Q, pool.dev, O)
    check(O, pool, Q, [0, 1, 2], 128 ** -0.5, 0, 0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_captured_step_follows_lengths_and_pages(Y, dtype, d):
    """One captured append + prefill + decode replays with other lengths, pages and row counts."""
    lens = [300, 20, 700]
    pool = Pool(Y, lens, 2, d, 16, dtype, room=64, rope=1e4)
    g = torch.Generator().manual_seed(4)
    R = 40
    k, v, q = (torch.randn(R, h, d, generator=g).to(DT[dtype]).cuda() for h in (2, 2, 6))
    cu = torch.tensor([0, 3, 3, 30], dtype=torch.int32, device="cuda")
    ws = torch.empty(Y.yoco_paged_attn_workspace_size(6, R, pool.dev), dtype=torch.uint8, device="cuda")

    def step(qo, o, od):
        Y.yoco_paged_append(k, v, pool.dev, cu, q=q, q_out=qo, workspace=ws)
        Y.yoco_paged_attn_prefill(qo, pool.dev, cu, o, window=100, sinks=2, workspace=ws)
        Y.yoco_paged_attn_decode(qo[:3], pool.dev, od, workspace=ws)

    mk = lambda: (torch.zeros(R, 6, d, dtype=DT[dtype], device="cuda"), torch.zeros(R, 6, d, dtype=DT[dtype], device="cuda"),  # noqa: E731
                  torch.zeros(3, 6, d, dtype=DT[dtype], device="cuda"))
    a, b = mk(), mk()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*a)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph, stream=side):
        step(*a)
    for new_lens, new_cu in (([300, 20, 700], [0, 3, 3, 30]), ([310, 60, 701], [0, 10, 39, 40]), ([5, 1, 730], [0, 5, 5, 5])):
        pool.dev.seq_lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        pool.dev.page_table.copy_(pool.dev.page_table.flip(0))
        cu.copy_(torch.tensor(new_cu, dtype=torch.int32))
        for x in a + b:
            x.zero_()
        # the flipped table may lack pages that the lengths need: reported, the same on both sides
        step(*b)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_streams_with_workspaces_of_their_own(Y):
    pools = [Pool(Y, [3000, 500 + i], 2, 128, 64, "bf16", seed=i) for i in range(2)]
    Qs = [torch.randn(2, 6, 128).bfloat16().cuda() for _ in range(2)]
    Os = [torch.empty_like(q) for q in Qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [torch.empty(Y.yoco_paged_attn_workspace_size(6, 2, p.dev), dtype=torch.uint8, device="cuda") for p in pools]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            Y.yoco_paged_attn_decode(Qs[i], pools[i].dev, Os[i], workspace=wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(Os[i], pools[i], Qs[i], [0, 1, 2], 128 ** -0.5, 0, 0)


def test_a_call_on_another_stream_keeps_its_own_workspace(Y):
    """Without a workspace the binding makes one; memory freed on the current stream must not be
    handed out again while the other stream still uses it."""
    pool = Pool(Y, [6000, 40], 2, 128, 64, "bf16")
    Q = torch.randn(2, 8, 128).bfloat16().cuda()
    want, side = torch.empty_like(Q), torch.cuda.Stream()
    Y.yoco_paged_attn_decode(Q, pool.dev, want)
    n = Y.yoco_paged_attn_workspace_size(8, 2, pool.dev)
    torch.cuda.synchronize()
    outs = [torch.empty_like(Q) for _ in range(8)]
    for o in outs:
        Y.yoco_paged_attn_decode(Q, pool.dev, o, stream=side)
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_results_do_not_change_from_call_to_call(Y):
    pool = Pool(Y, [5000, 30, 900], 2, 128, 64, "bf16")
    Q = torch.randn(3, 6, 128).bfloat16().cuda()
    outs = []
    for _ in range(3):
        O = torch.empty_like(Q)
        Y.yoco_paged_attn_decode(Q, pool.dev, O)
        outs.append(O)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_injected_failure_writes_nothing(Y):
    pool = Pool(Y, [100], 2, 128, 16, "bf16")
    Q = torch.randn(1, 4, 128).bfloat16().cuda()
    O = torch.full_like(Q, 3.0)
    Y._check(Y.lib.yoco_test_hook(Y.YOCO_HOOK_FAIL_NEXT_CALLS, 3), "hook")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    before = pool.dev.v.clone()
    for call in (lambda: Y.yoco_paged_attn_decode(Q, pool.dev, O), lambda: Y.yoco_paged_attn_prefill(Q, pool.dev, cu, O),
                 lambda: Y.yoco_paged_append(Q[:, :2].contiguous(), Q[:, :2].contiguous(), pool.dev)):
        with pytest.raises(Y.YocoError) as e:
            call()
        assert e.value.status == Y.YOCO_ERR_CUDA
    torch.cuda.synchronize()
    assert bool((O == 3.0).all()) and torch.equal(before.view(torch.int16), pool.dev.v.view(torch.int16))
