"""GPU checks of the rotary encoding with layouts, parts of a head and scaled frequencies, against
the formulas in 64 bits.

Bounds, element by element: p theta is off by p 2^-53 theta on either side for each of two roundings
(4 p 2^-53 in all), the angle by 2^-32 turns and its rounding to fp32 (2^-25 half turns: 1.6 u), cosine
and sine by 2 u each; with the magnitude and the products (u each)
|y - y64| <= h |y64| + (8 u + p 2^-51) mag (|x0| + |x1|), h half a step of the type, u = 2^-24.
"""
import math

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


def frequencies(r, base, scaling, factor, original, low, high):
    i = torch.arange(r // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    theta = torch.tensor(base, dtype=torch.float64) ** (-2 * i / r)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "by_parts":
        w = ((original * theta / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        theta = theta * (w + (1 - w) / factor)
    return theta


def turned(x, pos, r, layout, magnitude, theta):
    """(y, bound) in 64 bits."""
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    x = x.double().cpu()
    a = pos.double()[:, None, None] * theta
    c, s = torch.cos(a), torch.sin(a)
    i = (slice(0, r, 2), slice(1, r, 2)) if layout == "pairs" else (slice(0, r // 2), slice(r // 2, r))
    x0, x1 = x[..., i[0]], x[..., i[1]]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., i[0]], y[..., i[1]] = magnitude * (x0 * c - x1 * s), magnitude * (x0 * s + x1 * c)
    for k in i:
        tol[..., k] = half * y[..., k].abs() + (8 * U + pos.double().abs()[:, None, None] * 2.0 ** -51) * magnitude * (x0.abs() + x1.abs())
    return y, tol


def check(got, x, pos, d, **kw):
    r = kw.get("rotary_dim") or d
    f = dict(base=1e4, scaling="none", factor=1.0, original=8192.0, low=1.0, high=32.0)
    f.update({k: v for k, v in kw.items() if k in f})
    y, tol = turned(x, pos, r, kw.get("layout", "pairs"), kw.get("magnitude", 1.0), frequencies(r, **f))
    off = (got.double().cpu() - y).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=16.0, magnitude=1.25, original=4096.0, base=5e5),
            dict(scaling="by_parts", factor=2.0, low=0.5, high=4.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("dtype,d,r", [("bf16", 128, None), ("bf16", 128, 48), ("bf16", 64, 16), ("f32", 128, 64),
                                       ("f32", 64, None), ("f32", 128, 112)])
def test_rows_at_positions(Y, dtype, d, r, layout, kw):
    g = torch.Generator().manual_seed(1)
    pos = torch.cat((torch.randint(0, 1 << 20, (30,), generator=g), torch.tensor([0, 1, -1, -5000, (1 << 31) - 1, -(1 << 31), 1 << 20])))
    x = torch.randn(len(pos), 5, d, generator=g).to(DT[dtype])
    out = torch.full_like(x, 9.0).cuda()
    Y.yoco_rope_apply_scaled(x.cuda(), Y.Rope(rotary_dim=r, layout=layout, **kw), out=out, positions=pos.to(torch.int32).cuda())
    check(out, x, pos, d, rotary_dim=r, layout=layout, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("rows,H", [(0, 3), (1, 1), (3, 7), (700, 3), (5000, 2), (2, 300)])
def test_sizes_in_place_and_strided(Y, dtype, layout, rows, H):
    """Out of a fused projection into strided rows, and in place, with rows at pos0 + i."""
    g = torch.Generator().manual_seed(2)
    d, rope = 128, Y.Rope(rotary_dim=96, layout=layout)
    fused = torch.randn(rows, H + 2, d, generator=g).to(DT[dtype])
    dev = fused.cuda()
    wide = torch.full((H + 1, rows + 1, d), 3.0, dtype=DT[dtype], device="cuda")  # head-major rows
    out = wide.transpose(0, 1)[:rows, :H]
    Y.yoco_rope_apply_scaled(dev[:, 1:H + 1], rope, out=out, pos0=1000)
    assert torch.equal(dev.cpu(), fused)
    check(out, fused[:, 1:H + 1], torch.arange(rows) + 1000, d, rotary_dim=96, layout=layout)
    assert bool((wide[H] == 3).all()) and bool((wide[:, rows] == 3).all())
    Y.yoco_rope_apply_scaled(dev[:, 1:H + 1], rope, pos0=1000)
    assert torch.equal(dev[:, 1:H + 1], out)
    assert torch.equal(dev[:, 0].cpu(), fused[:, 0]) and torch.equal(dev[:, H + 1].cpu(), fused[:, H + 1])


def test_channels_that_do_not_turn_keep_their_bits(Y):
    x = torch.randn(4, 3, 64, device="cuda").to(torch.bfloat16)
    x[..., 32:] = float("inf")
    x[1, :, 40] = float("nan")
    out = torch.empty_like(x)
    for layout in ("pairs", "halves"):
        Y.yoco_rope_apply_scaled(x, Y.Rope(rotary_dim=32, layout=layout, magnitude=2.0, scaling="linear", factor=2.0), out=out, pos0=7)
        assert torch.equal(out[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
        assert bool(torch.isfinite(out[..., :32]).all())


def test_pairs_of_whole_heads_agree_with_the_plain_call(Y):
    x = torch.randn(1, 200, 4, 128, device="cuda")
    out = torch.empty(200, 4, 128, device="cuda")
    Y.yoco_rope_apply_scaled(x[0], Y.Rope(base=1e4), out=out, pos0=4000)
    want = x.clone()
    Y.yoco_rope_apply(want, 1e4, pos0=4000)
    # the plain call's angles carry the fp32 error of an offset below 32 besides: 32 * 2^-23 rad
    assert float((out - want[0]).abs().max()) <= (32 * 2.0 ** -23 + 16 * U) * 2 * float(x.abs().max())


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("kw", [dict(layout="halves", rotary_dim=32), dict(layout="halves", scaling="ntk", factor=4.0),
                                dict(layout="pairs", rotary_dim=48, scaling="by_parts", factor=8.0, magnitude=1.2)])
def test_append(Y, dtype, d, kw):
    """k turned into its slots, v copied, q turned, every other slot of the pool as it was."""
    g = torch.Generator().manual_seed(4)
    new, ctx, page, Hkv, Hq = [3, 0, 70, 1, 33], [0, 7, 29, 100, 500], 16, 2, 6
    lens = [a + b for a, b in zip(new, ctx)]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=g)
    table = torch.full((5, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    fused = torch.randn(cu[-1] + 2, Hq + 2 * Hkv, d, generator=g).to(DT[dtype])
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    pool = torch.full((len(order), Hkv, page, d), 5.0, dtype=DT[dtype])
    cache = Y.PagedKV(pool.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    dev = fused.cuda()
    out = torch.full((cu[-1] + 2, Hq, d), 5.0, dtype=DT[dtype], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    Y.yoco_paged_append_rope(dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], cache, Y.Rope(**kw),
                             cu_rows=torch.tensor(cu, dtype=torch.int32).cuda(), q=dev[:, :Hq], q_out=out, workspace=ws)
    Y.yoco_workspace_status(ws)
    kc, vc = cache.k.cpu(), cache.v.cpu()
    left = torch.ones(len(order), page, dtype=torch.bool)
    for b in range(5):
        rows, pos = slice(cu[b], cu[b + 1]), torch.arange(ctx[b], lens[b])
        ids = table[b].long()[pos // page]
        left[ids, pos % page] = False
        check(kc[ids, :, pos % page], k[rows], pos, d, **kw)
        assert torch.equal(vc[ids, :, pos % page], v[rows])
        check(out[rows], q[rows], pos, d, **kw)
    assert bool((kc.transpose(1, 2)[left] == 5).all()) and bool((vc.transpose(1, 2)[left] == 5).all())
    assert bool((out[cu[-1]:] == 5).all())


def test_append_one_row_per_sequence_and_q_alone(Y):
    B, d = 70, 64
    cache = Y.PagedKV(torch.zeros(B, 1, 16, d, device="cuda"), torch.zeros(B, 1, 16, d, device="cuda"),
                      torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                      torch.full((B,), 9, dtype=torch.int32, device="cuda"))
    x = torch.randn(B, 1, d)
    q = torch.randn(B, 4, d)
    qd = q.cuda()
    rope = Y.Rope(layout="halves", rotary_dim=32)
    Y.yoco_paged_append_rope(x.cuda(), x.cuda(), cache, rope)
    check(cache.k[:, :, 8], x, torch.full((B,), 8), d, rotary_dim=32, layout="halves")
    assert torch.equal(cache.v[:, :, 8].cpu(), x) and bool((cache.k[:, :, :8] == 0).all())
    Y.yoco_paged_append_rope(None, None, cache, rope, q=qd)
    check(qd, q, torch.full((B,), 8), d, rotary_dim=32, layout="halves")


def test_on_another_stream_and_in_a_graph(Y):
    x = torch.randn(100, 4, 128, device="cuda")
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    out, rope = torch.zeros_like(x), Y.Rope(layout="halves")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y.yoco_rope_apply_scaled(x, rope, out=out, positions=pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(out, x.cpu(), torch.arange(100), 128, layout="halves")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y.yoco_rope_apply_scaled(x, rope, out=out, positions=pos)
    pos += 1000
    g.replay()
    check(out, x.cpu(), torch.arange(100) + 1000, 128, layout="halves")


def test_binding_refuses_what_it_cannot_marshal(Y):
    x = torch.zeros(4, 2, 64, device="cuda")
    for bad in (dict(out=torch.zeros(4, 2, 64)), dict(out=torch.zeros(4, 3, 64, device="cuda")),
                dict(out=torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)),
                dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda")), dict(positions=torch.zeros(4, dtype=torch.int32)),
                dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(pos0=1 << 40)):
        with pytest.raises(ValueError):
            Y.yoco_rope_apply_scaled(x, Y.Rope(), **bad)
    with pytest.raises(ValueError):
        Y.yoco_rope_apply_scaled(x.transpose(1, 2), Y.Rope())
    with pytest.raises(TypeError):
        Y.yoco_rope_apply_scaled(x.half(), Y.Rope())
    with pytest.raises(Y.YocoError):  # a stride that is no multiple of 16 bytes
        Y.yoco_rope_apply_scaled(torch.zeros(4, 131, device="cuda")[:, :128].view(4, 2, 64), Y.Rope())
