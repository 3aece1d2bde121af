"""The page, rotary and scored calls together, as a server uses them: pages handed out on the device,
prompts appended with their rotation and read, forked, grown copy on write, cut back, moved together,
against a plain model that keeps every sequence's rows in a list of its own."""
import pytest
import torch

import test_gpu_paged_scored as S
import test_gpu_rope_scaled as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


class Dense:
    """What the cache holds: the sequences' rows as the pool has them."""

    def __init__(self, B, Hkv, d):
        self.lens, self.Hkv = [0] * B, Hkv
        self.k = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(B)]
        self.v = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(B)]

    def rows(self, b, hk):
        return self.k[b][:, hk], self.v[b][:, hk]


@pytest.mark.parametrize("dtype,d,Hq,Hkv,page,graph", [("bf16", 128, 6, 2, 16, False), ("f32", 64, 4, 4, 32, False), ("bf16", 128, 8, 1, 64, True)])
def test_serving_rounds(Y, dtype, d, Hq, Hkv, page, graph):
    B, pages, most = 6, 90 if page == 16 else 60, 40
    dt = R.DT[dtype]
    kw = dict(layout="halves", rotary_dim=d // 2, scaling="by_parts", factor=4.0)
    rope, slopes, prefix = Y.Rope(**kw), S.slopes_of(Hq), [20, 0, 7, 0, 0, 3]
    nan = torch.full((pages, Hkv, page, d), float("nan"), dtype=dt)
    cache = Y.PagedKV(nan.cuda(), nan.cuda(), torch.full((B, most), -1, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda())
    refs = torch.zeros(pages, dtype=torch.int32).cuda()
    pool_ws = torch.zeros(Y.yoco_paged_pool_workspace_size(cache), dtype=torch.uint8).cuda()
    scores = Y.PagedScores(12.0, slopes.cuda(), S.cuda_ints(prefix))
    want = Dense(B, Hkv, d)
    g = torch.Generator().manual_seed(9)

    def resize(new):
        Y.yoco_paged_resize(cache, refs, S.cuda_ints(new), workspace=pool_ws)
        for b, n in enumerate(new):
            if 0 <= n < want.lens[b]:
                want.k[b], want.v[b], want.lens[b] = want.k[b][:n], want.v[b][:n], n

    def round_of(new):
        """Grow by `new` rows each, append them, attend."""
        resize([want.lens[b] + t if t else -1 for b, t in enumerate(new)])
        cu = [0]
        for t in new:
            cu.append(cu[-1] + t)
        fused = torch.randn(cu[-1], Hq + 2 * Hkv, d, generator=g).to(dt)
        dev, one = fused.cuda(), all(t == 1 for t in new)
        q = torch.empty(cu[-1], Hq, d, dtype=dt, device="cuda")
        O = torch.zeros_like(q)
        at = S.cuda_ints(cu)
        ws = torch.zeros(Y.yoco_paged_attn_workspace_size(Hq, cu[-1], cache), dtype=torch.uint8).cuda()

        def calls():
            Y.yoco_paged_append_rope(dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], cache, rope, cu_rows=at, q=dev[:, :Hq], q_out=q, workspace=ws)
            if one:
                Y.yoco_paged_attn_decode_scored(q, cache, O, scores, workspace=ws)
            else:
                Y.yoco_paged_attn_prefill_scored(q, cache, at, O, scores, workspace=ws)
        if graph:
            calls()  # (what a call sets up once)
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded):
                calls()
            recorded.replay()
        else:
            calls()
        Y.yoco_workspace_status(ws)
        Y.yoco_workspace_status(pool_ws)
        for b, t in enumerate(new):
            rows, pos = slice(cu[b], cu[b + 1]), torch.arange(t) + want.lens[b]
            # the cache's own rounding of k is checked here, and the attention on what it holds
            table = cache.page_table[b].cpu().long()
            k, v = cache.k.cpu()[table[pos // page], :, pos % page], cache.v.cpu()[table[pos // page], :, pos % page]
            R.check(k, fused[rows, Hq:Hq + Hkv], pos, d, **kw)
            R.check(q[rows], fused[rows, :Hq], pos, d, **kw)
            assert torch.equal(v, fused[rows, Hq + Hkv:])
            want.k[b], want.v[b] = torch.cat((want.k[b], k.double())), torch.cat((want.v[b], v.double()))
            want.lens[b] += t
        S.check(O, want, q, cu, torch.zeros(cu[-1], dtype=torch.int64), prefix, 12.0, slopes, 0, 0, d ** -0.5)

    def fork(src, dst):
        Y.yoco_paged_fork(cache, refs, S.cuda_ints(src), S.cuda_ints(dst), workspace=pool_ws)
        for a, b in zip(src, dst):
            want.k[b], want.v[b], want.lens[b] = want.k[a], want.v[a], want.lens[a]

    round_of([50, 33, 0, 0, 70, 0])
    fork([0, 1, 0], [2, 3, 5])
    for _ in range(3):
        round_of([1] * B)
    resize([want.lens[0] - 5, 0, -1, 40, -1, 10])  # rolled back, ended
    Y.yoco_paged_compact(cache, refs, workspace=pool_ws)
    live = int((refs > 0).sum())
    assert bool((refs[:live] > 0).all()) and bool((refs[live:] == 0).all())
    round_of([7, 90, 1, 0, 3, 1])
    round_of([1] * B)
    resize([0] * B)
    Y.yoco_workspace_status(pool_ws)
    assert int(refs.abs().sum()) == 0 and bool((cache.page_table == -1).all())
