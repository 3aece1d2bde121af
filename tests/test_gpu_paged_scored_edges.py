"""GPU checks of the scored paged calls where positions are far or negative, against the definition in 64
bits, element by element.

Far positions: o = sum w v, so an error of e_m in the score of slot m moves o by at most
sum w_m e_m (|v_m| + |o|).  With u = 2^-24, d channels and n slots e_m is (d + 4) u S_m for the product
(S_m = scale sum |q_i k_i|), 8 u (|x_m| + B_m) for cap, bias B_m = slope |p - m| (the distance to fp32, the
slope times log2(e), the product, the sum) and exponential; the sums add 2 n u.  A distance that is
formed from two rounded numbers is off by whole slots there, far outside this.  Weights and outputs
rounded to bf16 are off by 2^-8 of themselves at most (tests/test_gpu_paged_scored.py).
"""
import math

import pytest
import torch

import test_gpu_paged as P
import test_gpu_paged_scored as S

pytestmark = pytest.mark.gpu

U = S.U
INT_MAX = 2147483647


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


def far_reference(k, v, slots, Q, pos, prefix, slopes, window, sinks, tensor, half):
    """k, v [n, Hkv, d] of the slots that are there; Q [T, Hq, d]."""
    T, Hq, d = Q.shape
    m, p = slots[None], pos[:, None]
    seen = ((m <= p) & ((m > p - window) | (m < sinks))) | (m < prefix)
    out, tol = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // k.shape[1])].double(), v[:, h // (Hq // k.shape[1])].double()
        q = Q[:, h].double()
        bias = float(slopes[h]) * (m - p).abs().double()
        x = q @ kh.T * d ** -0.5 - bias
        w = torch.softmax(x.masked_fill(~seen, -math.inf), 1)
        e = U * ((d + 4) * (q.abs() @ kh.abs().T * d ** -0.5) + 8 * (x.abs() + bias.abs()) + 2 * seen.sum(1, keepdim=True))
        we = w * (e + (2.0 ** -8 if tensor else 0.0))
        o = w @ vh
        out[:, h], tol[:, h] = o, half * o.abs() + we @ vh.abs() + we.sum(1, keepdim=True) * o.abs() + 1e-30
    return out, tol


@pytest.mark.parametrize("dtype,d", S.TYPES)
@pytest.mark.parametrize("page,prefix,length", [(16, 0, 2 ** 24 + 40), (32, 0, 2 ** 25 + 77), (16, 20, 2 ** 24 + 1000), (64, 0, 2 ** 26 + 5)])
def test_distances_past_24_bits(Y, dtype, d, page, prefix, length):
    """A long stream behind a window, its sinks' or prefix's slots in one step with the window's first:
    the entries between them name no page."""
    new, Hq, Hkv, window, sinks = 45, 6, 2, 32, 4
    front, back = -(-max(sinks, prefix) // page), (length - new - window) // page
    entries = list(range(front)) + list(range(back, -(-length // page)))
    g = torch.Generator().manual_seed(length + page)
    k, v = (torch.randn(len(entries), Hkv, page, d, generator=g).to(P.DT[dtype]) for _ in range(2))
    table = torch.full((1, entries[-1] + 1), -1, dtype=torch.int32)
    table[0, entries] = torch.arange(len(entries), dtype=torch.int32)
    cache = Y.PagedKV(k.cuda(), v.cuda(), table.cuda(), S.cuda_ints([length]))
    slots = (torch.tensor(entries)[:, None] * page + torch.arange(page)).reshape(-1)
    there = slots < length
    rows = [t.transpose(1, 2).reshape(-1, Hkv, d)[there] for t in (k, v)]
    slots = slots[there]
    slopes = torch.tensor([0.5, 0.05, 1e-7, 0.0, -1e-7, 2.0])
    scores = Y.PagedScores(slopes=slopes.cuda(), prefix=S.cuda_ints([prefix]))
    Q = (torch.randn(new, Hq, d, generator=g) * 2).to(P.DT[dtype])
    half = 2.0 ** -8 if dtype == "bf16" else U
    for decode in (False, True):
        q = Q[-1:] if decode else Q
        O = torch.empty_like(q, device="cuda")
        ws = torch.zeros(Y.yoco_paged_attn_workspace_size(Hq, q.shape[0], cache), dtype=torch.uint8, device="cuda")
        if decode:
            Y.yoco_paged_attn_decode_scored(q.cuda(), cache, O, scores, window=window, sinks=sinks, workspace=ws)
        else:
            Y.yoco_paged_attn_prefill_scored(q.cuda(), cache, S.cuda_ints([0, new]), O, scores, window=window, sinks=sinks,
                                             workspace=ws)
        Y.yoco_workspace_status(ws)
        tensor = dtype == "bf16" and (d == 128 or not decode)
        pos = torch.arange(length - q.shape[0], length)
        ref, tol = far_reference(*rows, slots, q, pos, prefix, slopes, window, sinks, tensor, half)
        off = (O.cpu().double() - ref).abs()
        assert torch.isfinite(off).all(), "not finite"
        worst = (off / tol).amax((0, 2))
        assert bool((worst <= 1.0).all()), (decode, worst.tolist())


@pytest.mark.parametrize("dtype,d", S.TYPES)
@pytest.mark.parametrize("mask", ["none", "prefix", "window", "cap", "bias", "all"])
@pytest.mark.parametrize("first", [0, INT_MAX, 1 << 30, -INT_MAX - 1])
def test_rows_before_the_first_slot(Y, dtype, d, mask, first):
    """Sequences with more new rows than slots (padding in front): rows at negative positions are zero,
    whatever their document start and the other rows' masks; some rows behind them see nothing either."""
    new, ctx = [200, 40, 3, 70], [-50, -3, -2, 30]
    lens = [a + b for a, b in zip(new, ctx)]
    kw = dict(none={}, prefix=dict(prefix=[150, 20, 1, 0]), window=dict(window=20, sinks=3), cap=dict(cap=15.0), bias=dict(bias=True),
              all=dict(cap=10.0, bias=True, window=30, sinks=2, prefix=[60, 7, 1, 50]))[mask]
    pos = torch.cat([torch.arange(c, n) for c, n in zip(ctx, lens)])
    doc = torch.where(pos < 0, first, 0)
    doc[120:130] = first
    _, _, O, _ = S.run(Y, new, ctx, 6, 2, d, 16, dtype, doc=doc, **kw)
    assert bool((O[:273][(pos[:273] < 0).cuda()] == 0).all())


@pytest.mark.parametrize("dtype,d", S.TYPES)
@pytest.mark.parametrize("first", [0, INT_MAX])
def test_rows_before_the_first_slot_of_cut_keys(Y, dtype, d, first):
    """The same where the keys are cut into pieces: a prefix makes every row block see all of them."""
    new, ctx = [2100], [-100]
    doc = torch.full((2100,), 0)
    doc[:100] = first
    doc[300:310] = first
    _, _, O, _ = S.run(Y, new, ctx, 2, 2, d, 64, dtype, doc=doc, prefix=[2000])
    assert bool((O[:100] == 0).all())


@pytest.mark.parametrize("dtype,d", S.TYPES)
def test_rows_of_empty_sequences(Y, dtype, d):
    """Sequences of length 0 with rows: zeros, beside one that is served."""
    pool = P.Pool(Y, [100, 0, 0], 2, d, 16, dtype)
    Q = (torch.randn(60, 6, d, generator=torch.Generator().manual_seed(2)) * 2).to(P.DT[dtype]).cuda()
    for first in (0, INT_MAX):
        O = torch.full_like(Q, 7.0)
        doc = torch.zeros(60, dtype=torch.int64)
        doc[20:] = first
        scores = Y.PagedScores(20.0, S.slopes_of(6).cuda(), S.cuda_ints([5, 1 << 30, 9]), S.cuda_ints(doc))
        Y.yoco_paged_attn_prefill_scored(Q, pool.dev, S.cuda_ints([0, 20, 50, 60]), O, scores, window=10, sinks=4)
        assert bool((O[20:] == 0).all())
        S.check(O[:20], pool, Q[:20], [0, 20, 20, 20], doc, [5, 0, 0], 20.0, S.slopes_of(6), 10, 4, d ** -0.5)
    O = torch.full((3, 6, d), 7.0, dtype=P.DT[dtype], device="cuda")
    Y.yoco_paged_attn_decode_scored(Q[:3], pool.dev, O, Y.PagedScores(20.0, prefix=S.cuda_ints([5, 1 << 30, 9])))
    assert bool((O[1:] == 0).all()) and bool((O[0] != 0).any())
