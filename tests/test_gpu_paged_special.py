"""GPU checks of the paged calls where values or metadata are not the ordinary ones: NaN and
infinities in queries and in slots that rows see, rows that see nothing, row bounds that fall
back, sequences' rows in several calls' order.

What a row gives is softmax's own answer: NaN where a score that it sees is NaN or +inf or where
all of them are -inf, the rest of the keys' answer where some are -inf, and zeros for a row at a
negative position, which sees nothing.  Finite answers are held to the bounds of
test_gpu_paged.py (its S taken over the slots of finite score: the others' weights are 0 on both
sides)."""
import itertools
import math

import pytest
import torch

import test_gpu_paged as P

pytestmark = pytest.mark.gpu
Y = P.Y  # the fixture

U, DT, TYPES = P.U, P.DT, P.TYPES


def answer(pool, q, b, pos, scale):
    """(o, bound, rows x heads that are NaN) in 64 bits of rows q [T, Hq, d] at positions pos."""
    T, Hq, d = q.shape
    out, tol = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    nan = torch.zeros(T, Hq, dtype=torch.bool)
    seen = torch.arange(pool.lens[b])[None] <= pos[:, None]
    n = seen.sum(1, keepdim=True)
    for h in range(Hq):
        k, v = pool.rows(b, h // (Hq // pool.Hkv))
        x = (q[:, h].double()[:, None, :] * k[None]).sum(-1) * scale if k.shape[0] <= 4096 else q[:, h].double() @ k.T * scale
        size = (q[:, h].double().abs() @ torch.where(torch.isfinite(k), k, 0.0).abs().T * scale)
        x = x.masked_fill(~seen, -math.inf)
        p = torch.softmax(x, 1)
        nan[:, h] = p.isnan().any(1) & (n[:, 0] > 0)
        p = torch.nan_to_num(p)
        S = torch.where(seen & torch.isfinite(x), size, 0.0).amax(1, keepdim=True)
        e32 = U * (2 * (d + 4) * S + 2 * n + 16)
        w, half = (2.0 ** -8 if d == 128 else 0.0, 2.0 ** -8) if q.dtype == torch.bfloat16 else (0.0, U)
        o = p @ v
        out[:, h], tol[:, h] = o, half * o.abs() + (e32 + w) * (p @ v.abs()) + 1e-30
    return out, tol, nan


def compare(got, pool, Q, cu, scale):
    got = got.cpu().double()
    some = False
    for b in range(len(pool.lens)):
        T = cu[b + 1] - cu[b]
        ref, tol, nan = answer(pool, Q[cu[b]:cu[b + 1]].cpu(), b, torch.arange(T) + pool.lens[b] - T, scale)
        mine = got[cu[b]:cu[b + 1]]
        assert torch.equal(mine.isnan().any(-1), nan), (b, int(mine.isnan().any(-1).sum()), int(nan.sum()))
        assert torch.equal(mine.isnan().all(-1), nan)
        off = ((mine - ref).abs() / tol).masked_fill(nan[..., None], 0.0)
        assert bool((off <= 1.0).all()), (b, float(off.max()))
        some |= bool(nan.any())
    return some


def queries(rows, Hq, d, dtype, seed):
    return (torch.randn(rows, Hq, d, generator=torch.Generator().manual_seed(seed)) * 2).to(DT[dtype])


def prefill(Y, pool, Q, cu):
    O = torch.full_like(Q, 7.0)
    Y.yoco_paged_attn_prefill(Q, pool.dev, torch.tensor(cu, dtype=torch.int32, device="cuda"), O)
    return O


def slots(pool, b, at):
    at = torch.as_tensor(at)
    return pool.table[b].long()[at // pool.page], at % pool.page


def put(pool, b, at, k, hk=slice(None), channel=slice(None)):
    """k into slots `at` of sequence b, on both sides."""
    pages, rows = slots(pool, b, at)
    for p, r in zip(pages.tolist(), rows.tolist()):
        pool.k[p, hk, r, channel] = k
    pool.dev.k.copy_(pool.k)


# few keys, and so many that the keys of these few rows are cut into pieces
CONTEXTS = [90, 9000]


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("ctx", CONTEXTS)
def test_prefill_of_a_nan_query_row(Y, dtype, d, ctx):
    pool = P.Pool(Y, [ctx + 5, 40], 2, d, 64, dtype)
    Q = queries(7, 6, d, dtype, 21)
    Q[2, 4, 3] = math.nan
    Q[6, 0] = math.nan
    Q = Q.cuda()
    assert compare(prefill(Y, pool, Q, [0, 5, 7]), pool, Q, [0, 5, 7], d ** -0.5)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("ctx", CONTEXTS)
@pytest.mark.parametrize("lo,hi", [(3, 4), (0, 700), (0, 768), (80, 93)])
def test_prefill_over_nan_keys(Y, dtype, d, ctx, lo, hi):
    """One NaN key, pieces of them (768 keys end where pieces of one, two or three tiles do), and
    keys that only the later rows see."""
    pool = P.Pool(Y, [ctx + 5, 40], 2, d, 64, dtype)
    lo, hi = min(lo, ctx), min(hi, ctx + 3)
    put(pool, 0, range(lo, hi), math.nan, hk=1)
    Q = queries(7, 6, d, dtype, 22).cuda()
    assert compare(prefill(Y, pool, Q, [0, 5, 7]), pool, Q, [0, 5, 7], d ** -0.5)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_prefill_of_chunks_with_a_nan_key_among_the_new_rows(Y, dtype, d):
    """Rows before the key's position are sound, those from it on are not."""
    pool = P.Pool(Y, [300, 140], 2, d, 64, dtype)
    put(pool, 0, [201], math.nan, hk=0)
    put(pool, 1, [139], math.nan)
    Q = queries(440, 6, d, dtype, 23).cuda()
    assert compare(prefill(Y, pool, Q, [0, 300, 440]), pool, Q, [0, 300, 440], d ** -0.5)


def decode(Y, pool, Q):
    O = torch.full_like(Q, 7.0)
    Y.yoco_paged_attn_decode(Q, pool.dev, O)
    return O


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("G", [1, 3, 16])
def test_decode_of_nan_queries_and_nan_keys(Y, dtype, d, G):
    """A NaN query; one NaN key among 1, 20 and 700; the first 64; all; the last."""
    pool = P.Pool(Y, [50, 1, 20, 700, 700, 130, 300, 70], 2, d, 16, dtype)
    for b, at in ((1, [0]), (2, [7]), (3, [3]), (4, range(64)), (5, range(130)), (6, [299])):
        put(pool, b, at, math.nan, hk=b % 2)
    Q = queries(8, 2 * G, d, dtype, 24)
    Q[0, G] = math.nan
    Q = Q.cuda()
    assert compare(decode(Y, pool, Q), pool, Q, list(range(9)), d ** -0.5)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("at", [range(5), range(4096), range(6000), range(8192), range(40000, 60001)])
def test_decode_of_a_long_sequence_with_nan_keys_is_nan(Y, dtype, d, at):
    """The runs that the keys are cut into (two tiles, four on the tensor cores) are NaN in part,
    from the first on, the first sixteen and no other, up to the last."""
    pool = P.Pool(Y, [60001], 1, d, 64, dtype)
    put(pool, 0, at, math.nan)
    Q = queries(1, 2, d, dtype, 25).cuda()
    assert bool(decode(Y, pool, Q).isnan().all())


@pytest.mark.parametrize("dtype,d", TYPES)
def test_decode_of_a_long_sequence_with_a_nan_query_is_nan(Y, dtype, d):
    pool = P.Pool(Y, [60001], 1, d, 64, dtype)
    Q = queries(1, 2, d, dtype, 26)
    Q[0, 1, 5] = math.nan
    Q = Q.cuda()
    O = decode(Y, pool, Q)
    assert bool(O[0, 1].isnan().all()) and bool(torch.isfinite(O[0, 0]).all())


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("n", [95, 9003, 60001])
def test_infinite_values_come_through(Y, dtype, d, n):
    """A value of +inf that a row sees makes its channel +inf, whole or cut, and no other."""
    pool = P.Pool(Y, [n], 1, d, 64, dtype)
    for m in (3, n // 2, n - 4):
        page, row = (int(x) for x in slots(pool, 0, m))
        pool.dev.v[page, 0, row, 5] = math.inf
    Q = queries(3, 2, d, dtype, 30).cuda() * 0.1
    for O in (prefill(Y, pool, Q, [0, 3]), decode(Y, pool, Q[:1].contiguous())):
        assert bool((O[..., 5] == math.inf).all())
        O[..., 5] = 0
        assert bool(torch.isfinite(O).all())


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("length,rows", [(10, 25), (2900, 2917)])
def test_rows_that_see_nothing_are_zeros_whatever_the_others_see(Y, dtype, d, length, rows):
    """More new rows than the sequence holds, in one block with rows whose values are NaN."""
    pool = P.Pool(Y, [length], 2, d, 16, dtype)
    pages, at = slots(pool, 0, range(min(length, 40)))
    for p, r in zip(pages.tolist(), at.tolist()):
        pool.dev.v[p, :, r] = math.nan
    Q = queries(rows, 6, d, dtype, 29).cuda()
    O = prefill(Y, pool, Q, [0, rows])
    assert bool((O[:rows - length] == 0).all()) and bool(O[rows - length:].isnan().all())


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("ctx", CONTEXTS)
@pytest.mark.parametrize("keys", ["all", "first", "last"])
def test_scores_of_minus_infinity(Y, dtype, d, ctx, keys):
    """Keys of score -inf have the weight 0; where a row sees no others there is no softmax."""
    n = ctx + 3
    pool = P.Pool(Y, [n, 10], 1, d, 64, dtype)
    at = {"all": range(n), "first": range(n - 60), "last": range(n - 60, n)}[keys]
    put(pool, 0, at, -math.inf, channel=2)
    Q = queries(5, 3, d, dtype, 27)
    Q[:, :, 2] = 1.0
    Q = Q.cuda()
    assert compare(prefill(Y, pool, Q, [0, 3, 5]), pool, Q, [0, 3, 5], d ** -0.5) == (keys == "all")
    Q = Q[:2].contiguous()
    assert compare(decode(Y, pool, Q), pool, Q, [0, 1, 2], d ** -0.5) == (keys == "all")


@pytest.mark.parametrize("dtype,d", TYPES)
def test_scores_of_plus_infinity_are_nan(Y, dtype, d):
    pool = P.Pool(Y, [95, 9003], 1, d, 64, dtype)
    for b in range(2):
        put(pool, b, [41], math.inf, channel=2)
    Q = queries(4, 3, d, dtype, 28)
    Q[:, :, 2] = 1.0
    Q = Q.cuda()
    assert bool(prefill(Y, pool, Q, [0, 2, 4]).isnan().all())
    assert bool(decode(Y, pool, Q[:2].contiguous()).isnan().all())


# ------------------------------------------------------- row bounds that fall back

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("more", [0, 37])
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 5, -1, 8], [0, 5, 3, 12], [0, 4, 100, 12], [2, 7, 7, 5], [-1, 3, 9, 12],
                                [0, 2 ** 31 - 1, 4, 9], [4, 2, 0, 3]])
def test_append_leaves_out_only_sequences_of_bad_bounds(Y, dtype, d, more, cu):
    """A sequence whose bounds decrease or leave [0, rows] has no rows; every other one is written,
    with a row that two of them claim in both caches and its q turned for the first."""
    rows, Hkv, Hq, page = 12, 2, 4, 16
    cu = cu + [cu[-1]] * more  # sequences without rows behind them: more than a warp looks up at once
    B = len(cu) - 1
    pool = P.Pool(Y, [60 + 3 * b for b in range(B)], Hkv, d, page, dtype, rope=1e4)
    g = torch.Generator().manual_seed(31)
    k, v, q = (torch.randn(rows, h, d, generator=g).to(DT[dtype]) for h in (Hkv, Hkv, Hq))
    k0, v0 = pool.dev.k.cpu(), pool.dev.v.cpu()
    out = torch.full((rows, Hq, d), 9.0, dtype=DT[dtype], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    Y.yoco_paged_append(k.cuda(), v.cuda(), pool.dev, torch.tensor(cu, dtype=torch.int32, device="cuda"), q=q.cuda(),
                        q_out=out, workspace=ws)
    assert P.status(Y, ws) == Y.YOCO_ERR_INVALID_ARG
    k1, v1, out = pool.dev.k.cpu(), pool.dev.v.cpu(), out.cpu()
    owner = [-1] * rows
    for b in range(B):
        c0, c1 = cu[b], cu[b + 1]
        if not 0 <= c0 <= c1 <= rows:
            continue
        for i in range(c0, c1):
            pos = pool.lens[b] - (c1 - c0) + i - c0
            pg, r = int(pool.table[b, pos // page]), pos % page
            P.close_turn(k1[pg, :, r][None], k[i:i + 1], torch.tensor([pos]), 1e4, dtype)
            assert torch.equal(v1[pg, :, r], v[i])
            k0[pg, :, r], v0[pg, :, r] = k1[pg, :, r], v1[pg, :, r]
            if owner[i] < 0:
                owner[i] = b
                P.close_turn(out[i:i + 1], q[i:i + 1], torch.tensor([pos]), 1e4, dtype)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(k0.view(bits), k1.view(bits)) and torch.equal(v0.view(bits), v1.view(bits))
    for i in range(rows):
        assert owner[i] >= 0 or bool((out[i] == 9.0).all())


# ------------------------------------------------------------------- streams

def test_own_workspace_on_another_stream_waits_for_nothing_of_the_current_one(Y):
    """Memory freed on the current stream, with the work that fills it still queued there, is not
    what a call on another stream gets for its workspace."""
    pool = P.Pool(Y, [6000, 40], 2, 128, 64, "bf16")
    Q, cu = queries(12, 8, 128, "bf16", 33).cuda(), torch.tensor([0, 7, 12], dtype=torch.int32, device="cuda")
    want, want_d, side = torch.empty_like(Q), torch.empty_like(Q[:2]), torch.cuda.Stream()
    Y.yoco_paged_attn_prefill(Q, pool.dev, cu, want)
    Y.yoco_paged_attn_decode(Q[:2], pool.dev, want_d)
    n = Y.yoco_paged_attn_workspace_size(8, 12, pool.dev)
    outs = [(torch.empty_like(Q), torch.empty_like(Q[:2])) for _ in range(4)]
    torch.cuda.synchronize()
    for o, od in outs:
        torch.cuda._sleep(4_000_000)  # a few milliseconds
        for _ in range(2):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        Y.yoco_paged_attn_prefill(Q, pool.dev, cu, o, stream=side)
        Y.yoco_paged_attn_decode(Q[:2], pool.dev, od, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(od, want_d) for o, od in outs)


def test_a_warp_gives_up_a_wait_as_one(Y):
    """Half a warp waits for what is complete, half for what never is (50 ms): none goes on."""
    ws = torch.full((64,), -1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert Y.lib.yoco_selftest_wait_timeout(ws.data_ptr(), 50_000_000, stream) == Y.YOCO_OK
    with pytest.raises(Y.YocoError) as e:
        Y.yoco_workspace_status(ws)
    assert e.value.status == Y.YOCO_ERR_TIMEOUT
    assert ws[1].item() == 0


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("few", [True, False])
def test_outputs_of_one_call_as_the_queries_of_the_next(Y, dtype, d, few):
    """Calls one behind the other, each starting while the one before it ends: what they give is what
    they give with the GPU waited for in between."""
    new = [1, 1, 1] if few else [60, 3, 130]
    lens = [700 + new[0], 3000 + new[1], 20 + new[2]]
    pool = P.Pool(Y, lens, 2, d, 64, dtype)
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device="cuda")
    Q = queries(sum(new), 6, d, dtype, 34).cuda()
    ws = torch.empty(Y.yoco_paged_attn_workspace_size(6, sum(new), pool.dev), dtype=torch.uint8, device="cuda")

    def chain(wait):
        outs = [Q]
        for i in range(12):
            O = torch.full_like(Q, math.nan)
            outs.append(O)
        torch.cuda.synchronize()
        for q, o in itertools.pairwise(outs):
            if few:
                Y.yoco_paged_attn_decode(q, pool.dev, o, scale=8.0, workspace=ws)
            else:
                Y.yoco_paged_attn_prefill(q, pool.dev, cu, o, scale=8.0, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        return torch.stack(outs[1:]).cpu()

    want = chain(True)
    assert bool(torch.isfinite(want).all())
    for _ in range(3):
        assert torch.equal(chain(False), want)


# ---------------------------------------------------------------- the work list

def work_list(ws):
    """(sequence, rows, tiles) of every entry that a prefill's plan left in the workspace: a count
    at byte 128, entries of 16 words (sequence, first row, rows, position, first and last tile)."""
    words = ws.cpu().view(torch.int32)
    n = int(words[32])
    e = words[64:64 + 16 * n].reshape(n, 16).tolist()
    return [(x[0], x[2], x[5] - x[4]) for x in e]


@pytest.mark.parametrize("B", [3, 40])
def test_window_plan_takes_the_longest_row_blocks_first(Y, B):
    """One query head to a kv head, so blocks of 256 rows, and a window of 20: prompts of 1025 rows have
    full blocks that see 275 slots and up to 15 of their first page, three tiles, and a last block
    that sees one; the others have a block of two tiles."""
    n = [1025 if b % 3 == 1 else 150 + b for b in range(B)]
    pool = P.Pool(Y, [2000 + t for t in n], 1, 128, 16, "bf16")
    cu = [0] + list(itertools.accumulate(n))
    Q = queries(cu[-1], 1, 128, "bf16", 35).cuda()
    O = torch.empty_like(Q)
    ws = torch.zeros(Y.yoco_paged_attn_workspace_size(1, cu[-1], pool.dev), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_attn_prefill(Q, pool.dev, torch.tensor(cu, dtype=torch.int32, device="cuda"), O, window=20, workspace=ws)
    Y.yoco_workspace_status(ws)
    P.check(O, pool, Q, cu, 128 ** -0.5, 20, 0)
    longest = {}  # of each sequence, in the order of the list
    for b, rows, tiles in work_list(ws):
        if rows:
            longest[b] = max(longest.get(b, 0), tiles)
    order = list(longest.values())
    assert len(order) == B and order == sorted(order, reverse=True) and set(order) == {2, 3}


def test_windows_and_sinks_past_32_bits(Y):
    """A window that no sequence reaches the end of, as a number that does not fit an int; likewise
    sinks, and numbers below any int."""
    pool = P.Pool(Y, [300, 77], 2, 128, 64, "bf16")
    Q, cu = queries(2, 4, 128, "bf16", 36).cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for call in (lambda O, **kw: Y.yoco_paged_attn_decode(Q, pool.dev, O, **kw),
                 lambda O, **kw: Y.yoco_paged_attn_prefill(Q, pool.dev, cu, O, **kw)):
        want, got = torch.empty_like(Q), torch.empty_like(Q)
        call(want)
        for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=20, sinks=2 ** 32 + 1)):
            call(got.fill_(math.nan), **kw)
            assert torch.equal(got, want)
        for kw in (dict(window=-2 ** 32 + 5), dict(window=7, sinks=-2 ** 32)):
            with pytest.raises(Y.YocoError) as e:
                call(got, **kw)
            assert e.value.status == Y.YOCO_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("B", [3, 300])
def test_prefill_results_do_not_change_from_call_to_call(Y, dtype, d, B):
    """Entries are taken from a counter and, of many sequences, ordered by atomics: what comes out is
    the same bit for bit."""
    new = [1 + (37 * b) % 90 for b in range(B)]
    pool = P.Pool(Y, [t + (53 * b) % 400 + (9000 if b == 1 else 0) for b, t in enumerate(new)], 2, d, 16, dtype)
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device="cuda")
    Q = queries(sum(new), 6, d, dtype, 37).cuda()
    outs = []
    for _ in range(5):
        outs.append(torch.full_like(Q, math.nan))
        Y.yoco_paged_attn_prefill(Q, pool.dev, cu, outs[-1])
    assert bool(torch.isfinite(outs[0]).all()) and all(torch.equal(outs[0], o) for o in outs[1:])
