"""GPU checks of the page calls against a plain model on the host: tables, counts, lengths and lists
exactly, the pools' contents bit by bit."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


class Model:
    """What the calls are documented to do, sequence by sequence."""

    def __init__(self, B, pages, page):
        self.page, self.B = page, B
        self.table, self.lens, self.refs = [[] for _ in range(B)], [0] * B, [0] * pages
        self.moves = []

    def held(self, n):
        return -(-n // self.page)

    def resize(self, new):
        P = self.page
        new = [self.lens[b] if n < 0 else n for b, n in enumerate(new)]
        for b, n in enumerate(new):
            if n < self.lens[b]:
                for p in self.table[b][self.held(n):]:
                    self.refs[p] -= 1
                del self.table[b][self.held(n):]
                self.lens[b] = n
        grow = [b for b in range(self.B) if new[b] > self.lens[b]]
        shared = {}
        for b in grow:
            if self.lens[b] % P and self.refs[self.table[b][-1]] > 1:
                shared.setdefault(self.table[b][-1], []).append(b)
        copies = sorted(b for p, who in shared.items() for b in (who[1:] if len(who) == self.refs[p] else who))
        need = sum(self.held(new[b]) - self.held(self.lens[b]) for b in grow) + len(copies)
        refs = list(self.refs)
        for b in copies:
            refs[self.table[b][-1]] -= 1
        free = [p for p, n in enumerate(refs) if n == 0]
        self.moves = []
        if need > len(free):
            self.free = len(free)
            return False
        self.refs, self.free, at = refs, len(free) - need, iter(free)
        for b in grow:
            if b in copies:
                p = next(at)
                self.moves.append((self.table[b][-1], p, self.lens[b] % P))
                self.table[b][-1] = p
                self.refs[p] = 1
            while len(self.table[b]) < self.held(new[b]):
                p = next(at)
                self.table[b].append(p)
                self.refs[p] = 1
            self.lens[b] = new[b]
        return True

    def fork(self, src, dst):
        ok = True
        pairs = []
        for i, (a, b) in enumerate(zip(src, dst)):
            good = 0 <= a < self.B and 0 <= b < self.B and a not in dst and b not in dst[:i] and self.lens[b] == 0
            ok = ok and good
            pairs += [(a, b)] if good else []
        for a, b in pairs:
            self.table[b], self.lens[b] = list(self.table[a]), self.lens[a]
            for p in self.table[a]:
                self.refs[p] += 1
        return ok

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        src = [p for p, n in enumerate(self.refs) if n and p >= live]
        dst = [p for p, n in enumerate(self.refs) if not n and p < live]
        to = dict(zip(src, dst))
        self.moves, self.free = [(a, b, self.page) for a, b in zip(src, dst)], live
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]


class Pair:
    """A model and the device's state, side by side."""

    def __init__(self, Y, B, pages, page, most, Hkv=2, d=64, dtype=torch.float32):
        self.Y, self.m = Y, Model(B, pages, page)
        self.k = torch.randn(pages, Hkv, page, d).to(dtype)
        self.v = torch.randn(pages, Hkv, page, d).to(dtype)
        self.cache = Y.PagedKV(self.k.cuda(), self.v.cuda(), torch.full((B, most), -1, dtype=torch.int32).cuda(),
                               torch.zeros(B, dtype=torch.int32).cuda())
        # another layer's pool, which follows by the lists
        self.layer = Y.PagedKV(self.k.cuda(), self.v.cuda(), self.cache.page_table, self.cache.seq_lens)
        self.refs = torch.zeros(pages, dtype=torch.int32).cuda()
        self.ws = torch.full((Y.yoco_paged_pool_workspace_size(self.cache),), 0xA5, dtype=torch.uint8).cuda()
        self.moves = torch.full((max(B, pages // 2) + 1, 4), 77, dtype=torch.int32).cuda()

    def resize(self, new, status=None):
        fits = self.m.resize(new)
        assert fits == (status is None)
        self.Y.yoco_paged_resize(self.cache, self.refs, torch.tensor(new, dtype=torch.int32).cuda(), moves=self.moves, workspace=self.ws)
        self.after(status)

    def fork(self, src, dst, status=None):
        self.m.fork(src, dst)
        self.m.moves = None
        self.Y.yoco_paged_fork(self.cache, self.refs, torch.tensor(src, dtype=torch.int32).cuda(),
                               torch.tensor(dst, dtype=torch.int32).cuda(), workspace=self.ws)
        self.after(status)

    def compact(self):
        self.m.compact()
        self.Y.yoco_paged_compact(self.cache, self.refs, moves=self.moves, workspace=self.ws)
        self.after(None)

    def after(self, status):
        if status is None:
            self.Y.yoco_workspace_status(self.ws)
        else:
            with pytest.raises(self.Y.YocoError) as e:
                self.Y.yoco_workspace_status(self.ws)
            assert e.value.status == status
        m = self.m
        assert self.cache.seq_lens.tolist() == m.lens
        assert self.refs.tolist() == m.refs
        for row, want in zip(self.cache.page_table.tolist(), m.table):
            assert row == want + [-1] * (len(row) - len(want))
        if m.moves is None:
            return
        moves = self.moves[:len(m.moves) + 1].tolist()
        assert moves[0] == [len(m.moves), m.free, 0, 0]
        assert [tuple(x) for x in moves[1:]] == [(a, b, n, 0) for a, b, n in m.moves]
        k, v = self.k.clone(), self.v.clone()
        for a, b, n in m.moves:
            k[b, :, :n], v[b, :, :n] = self.k[a, :, :n], self.v[a, :, :n]
        self.k, self.v = k, v
        self.Y.yoco_paged_copy(self.layer, self.moves)
        for c in (self.cache, self.layer):
            assert torch.equal(c.k.cpu(), k) and torch.equal(c.v.cpu(), v)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("B,pages,page,most,Hkv,d,dtype", [
    (1, 5, 16, 8, 1, 64, torch.float32), (7, 40, 16, 20, 2, 64, torch.bfloat16), (60, 300, 32, 30, 1, 128, torch.bfloat16),
    (1100, 5000, 16, 12, 1, 64, torch.bfloat16), (20, 9000, 16, 300, 1, 64, torch.bfloat16),
    (12, 25, 1024, 6, 1, 64, torch.float32)])
def test_random_rounds(Y, B, pages, page, most, Hkv, d, dtype, seed):
    rng = random.Random(seed)
    s = Pair(Y, B, pages, page, most, Hkv, d, dtype)
    top = min(most, 3 * pages // B + 1) * page
    for step in range(14):
        what = rng.choice(["resize", "resize", "resize", "fork", "compact"])
        m = s.m
        if what == "resize":
            new = [rng.choice([-1, n, 0, rng.randrange(n + 1), min(n + rng.randrange(40), most * page), rng.randrange(top)])
                   for n in m.lens]
            probe = Model(B, pages, page)
            probe.table, probe.lens, probe.refs = [list(r) for r in m.table], list(m.lens), list(m.refs)
            s.resize(new, None if probe.resize(new) else Y.YOCO_ERR_CAPACITY)
        elif what == "fork":
            empty = [b for b in range(B) if m.lens[b] == 0]
            full = [b for b in range(B) if m.lens[b]]
            if empty and full:
                dst = rng.sample(empty, rng.randint(1, len(empty)))
                s.fork([rng.choice(full) for _ in dst], dst)
        else:
            s.compact()


def test_the_first_of_those_that_all_grow_keeps_the_page(Y):
    s = Pair(Y, 6, 40, 16, 8)
    s.resize([0, 20, 0, 0, 5, 0])
    s.fork([1, 1, 4], [0, 2, 5])
    s.resize([21, 25, 40, 0, 5, 6])  # 0, 1, 2 share and grow: 0 keeps; 4 stays, 5 copies
    assert [m[2] for m in s.m.moves] == [4, 4, 5]
    s.resize([3, 3, 3, 0, 3, 3])
    s.resize([-1, 4, -1, 7, -1, -1])
    s.fork([1, 3], [0, 2], status=Y.YOCO_ERR_INVALID_ARG)


def test_a_call_without_room_changes_nothing_but_what_shrinks(Y):
    s = Pair(Y, 4, 6, 16, 8)
    s.resize([30, 40, 0, 0])
    s.fork([0], [2])
    s.resize([31, 17, 60, 100], status=Y.YOCO_ERR_CAPACITY)
    s.resize([31, 0, 31, 0])  # both share the page: one copy
    s.resize([128, 128, 128, 128], status=Y.YOCO_ERR_CAPACITY)
    s.resize([0, 0, 0, 96])
    s.resize([1, -1, -1, -1], status=Y.YOCO_ERR_CAPACITY)


def test_needs_past_32_bits_are_no_room(Y):
    B = 4096
    k = torch.zeros(8, 1, 16, 64, device="cuda")
    # a table this wide is never touched where there is no room for it
    table = torch.full((B, 1 << 20), -1, dtype=torch.int32, device="cuda")
    cache = Y.PagedKV(k, k, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    refs = torch.zeros(8, dtype=torch.int32, device="cuda")
    ws = torch.zeros(Y.yoco_paged_pool_workspace_size(cache), dtype=torch.uint8, device="cuda")
    Y.yoco_paged_resize(cache, refs, torch.full((B,), 1 << 24, dtype=torch.int32, device="cuda"), workspace=ws)
    with pytest.raises(Y.YocoError) as e:
        Y.yoco_workspace_status(ws)
    assert e.value.status == Y.YOCO_ERR_CAPACITY
    assert int(refs.abs().sum()) == 0 and int(cache.seq_lens.sum()) == 0


def test_entries_past_32_bits_go_back(Y):
    """2100 forks of a sequence of 2^20 pages: 2^31 and more table entries are given back in one call."""
    B, n = 2100, 1 << 20
    k = torch.zeros(n + 5, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = Y.PagedKV(k, k, torch.full((B, n), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"))
    refs = torch.zeros(n + 5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(Y.yoco_paged_pool_workspace_size(cache), dtype=torch.uint8, device="cuda")
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    lens[7] = 16 * n
    Y.yoco_paged_resize(cache, refs, lens, workspace=ws)
    dst = torch.tensor([b for b in range(B) if b != 7], dtype=torch.int32, device="cuda")
    Y.yoco_paged_fork(cache, refs, torch.full_like(dst, 7), dst, workspace=ws)
    Y.yoco_workspace_status(ws)
    assert bool((refs[:n] == B).all()) and bool((refs[n:] == 0).all())
    lens.fill_(0)
    lens[B - 1] = 16 * n - 16  # all but the last page of the last one
    Y.yoco_paged_resize(cache, refs, lens, workspace=ws)
    Y.yoco_workspace_status(ws)
    assert bool((refs[:n - 1] == 1).all()) and bool((refs[n - 1:] == 0).all())
    assert bool((cache.page_table[:B - 1] == -1).all()) and int(cache.page_table[B - 1, n - 1]) == -1


def test_bad_forks_are_left_out(Y):
    s = Pair(Y, 8, 40, 16, 8)
    s.resize([20, 30, 40, 0, 0, 0, 0, 0])
    s.fork([0, 1, 0, 9, 0, -1, 3, 2], [3, 3, 1, 4, 8, 5, 6, 7], status=Y.YOCO_ERR_INVALID_ARG)
    assert s.m.lens == [20, 30, 40, 20, 0, 0, 0, 40]


def test_bad_lengths_entries_and_counts_are_recorded(Y):
    def fresh():
        s = Pair(Y, 3, 20, 16, 4)
        s.resize([20, 33, 7])
        return s

    def bad(call):
        s = fresh()
        call(s)
        torch.cuda.synchronize()
        with pytest.raises(Y.YocoError) as e:
            Y.yoco_workspace_status(s.ws)
        assert e.value.status == Y.YOCO_ERR_INVALID_ARG
        return s

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def too_long(s):
        Y.yoco_paged_resize(s.cache, s.refs, ints(-1, 65, 20), workspace=s.ws)
    s = bad(too_long)
    assert s.cache.seq_lens.tolist() == [20, 33, 20]  # the others are served

    def bad_len(s):
        s.cache.seq_lens[0] = 1000
        Y.yoco_paged_resize(s.cache, s.refs, ints(0, 0, 20), workspace=s.ws)
    s = bad(bad_len)
    assert s.cache.seq_lens.tolist() == [1000, 0, 20]

    def bad_entry(s):
        s.cache.page_table[1, 1] = 12345
        Y.yoco_paged_resize(s.cache, s.refs, ints(-1, 0, -1), workspace=s.ws)
    s = bad(bad_entry)
    assert int(s.refs.sum()) == 3 + 1  # the page that no entry names stays counted

    def low_count(s):
        s.refs.zero_()
        Y.yoco_paged_resize(s.cache, s.refs, ints(-1, 0, -1), workspace=s.ws)
    s = bad(low_count)
    assert int(s.refs.abs().sum()) == 0

    def not_counted(s):
        s.refs.zero_()
        Y.yoco_paged_compact(s.cache, s.refs, workspace=s.ws)
    bad(not_counted)

    def fork_bad_len(s):
        s.cache.seq_lens[1] = -4
        s.cache.seq_lens[2] = 0
        Y.yoco_paged_fork(s.cache, s.refs, ints(1), ints(2), workspace=s.ws)
    bad(fork_bad_len)


def test_pages_that_a_window_has_left(Y):
    """Entries of -1 in front are passed over by every call, and stay -1."""
    def ints(*x):
        return torch.tensor(x, dtype=torch.int32).cuda()
    s = Pair(Y, 4, 30, 16, 8)
    s.resize([60, 100, 0, 0])
    for e in (0, 1, 2):  # given back by the caller
        s.refs[s.m.table[1][e]] -= 1
    s.cache.page_table[1, :3] = -1
    Y.yoco_paged_fork(s.cache, s.refs, ints(1), ints(2), workspace=s.ws)
    Y.yoco_paged_resize(s.cache, s.refs, ints(0, 101, 110, 20), workspace=s.ws)
    Y.yoco_paged_compact(s.cache, s.refs, workspace=s.ws)
    Y.yoco_workspace_status(s.ws)
    table = s.cache.page_table.cpu()
    assert table[1, :3].tolist() == table[2, :3].tolist() == [-1] * 3
    pages = [p for row in table.tolist() for p in row if p >= 0]
    # 4 pages of sequence 1, of which 3 are sequence 2's too; its copy of the fourth; 2 of sequence 3
    assert sorted(set(pages)) == list(range(7)) and int((s.refs > 0).sum()) == 7
    assert s.refs.tolist() == [pages.count(p) for p in range(30)]
    Y.yoco_paged_resize(s.cache, s.refs, ints(0, 0, 0, 0), workspace=s.ws)
    Y.yoco_workspace_status(s.ws)
    assert int(s.refs.abs().sum()) == 0


def test_large_pool(Y):
    """More pages than a pass of the warps' runs takes at once, handed out and moved across all of them."""
    pages, page, most = 400000, 16, 5000
    k = torch.zeros(pages, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    k[:, 0, 0, 0] = torch.arange(pages, device="cuda").remainder(256).to(torch.bfloat16)
    cache = Y.PagedKV(k, k.clone(), torch.full((100, most), -1, dtype=torch.int32).cuda(), torch.zeros(100, dtype=torch.int32).cuda())
    refs = torch.zeros(pages, dtype=torch.int32).cuda()
    ws = torch.zeros(Y.yoco_paged_pool_workspace_size(cache), dtype=torch.uint8).cuda()
    Y.yoco_paged_resize(cache, refs, torch.full((100,), 4000 * page - 3, dtype=torch.int32).cuda(), workspace=ws)
    assert torch.equal(cache.page_table[:, :4000].reshape(-1), torch.arange(pages, dtype=torch.int32, device="cuda"))
    low = torch.where(torch.arange(100) % 3 == 1, 0, -1).to(torch.int32).cuda()
    Y.yoco_paged_resize(cache, refs, low, workspace=ws)
    kept = (torch.arange(100, device="cuda") % 3 != 1).nonzero()[:, 0]
    marks = cache.page_table[kept, :4000].long().remainder(256)
    Y.yoco_paged_compact(cache, refs, workspace=ws)
    Y.yoco_workspace_status(ws)
    n = len(kept) * 4000
    now = cache.page_table[kept, :4000].long()
    assert torch.equal(now.reshape(-1).sort()[0], torch.arange(n, device="cuda"))
    assert bool((refs[:n] == 1).all()) and bool((refs[n:] == 0).all())
    for t in (cache.k, cache.v):
        assert torch.equal(t[now, 0, 0, 0].long(), marks)
    Y.yoco_paged_resize(cache, refs, torch.full((100,), 4000 * page, dtype=torch.int32).cuda(), workspace=ws)
    Y.yoco_workspace_status(ws)
    assert bool((refs == 1).all())
    assert torch.equal(cache.page_table[:, :4000].reshape(-1).sort()[0], torch.arange(pages, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_pools_past_32_bits_of_elements(Y, dtype, d):
    """Pages behind 2^31 elements of each tensor: appended to with a rotation, shared, copied, attended, moved."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    lead = 2 ** 31 // (2 * 64 * d)
    g = torch.Generator().manual_seed(9)

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def served(first):
        """Pages before `first` are someone else's.  What every call gives, and where it was."""
        k, v = (torch.empty(first + 9, 2, 64, d, dtype=t, device="cuda") for _ in range(2))
        k[first:], v[first:] = 0, 0
        cache = Y.PagedKV(k, v, torch.full((3, 4), -1, dtype=torch.int32).cuda(), ints(0, 0, 0))
        refs = torch.zeros(first + 9, dtype=torch.int32, device="cuda")
        refs[:first] = 1
        ws = torch.zeros(Y.yoco_paged_pool_workspace_size(cache), dtype=torch.uint8, device="cuda")
        Y.yoco_paged_resize(cache, refs, ints(150, 0, 40), workspace=ws)
        rope = Y.Rope(layout="halves", rotary_dim=32, scaling="ntk", factor=4.0)
        Y.yoco_paged_append_rope(new[0], new[1], cache, rope, cu_rows=ints(0, 150, 150, 190), workspace=ws)
        Y.yoco_paged_fork(cache, refs, ints(0), ints(1), workspace=ws)
        Y.yoco_paged_resize(cache, refs, ints(151, 200, 41), workspace=ws)
        rows = new[2][:52]
        Y.yoco_paged_append_rope(rows, rows, cache, rope, cu_rows=ints(0, 1, 51, 52), workspace=ws)
        out = [torch.zeros(52, 6, d, dtype=t, device="cuda"), torch.zeros(3, 6, d, dtype=t, device="cuda")]
        scores = Y.PagedScores(softcap=30.0)
        Y.yoco_paged_attn_prefill_scored(q, cache, ints(0, 1, 51, 52), out[0], scores)
        Y.yoco_paged_attn_decode_scored(q[:3], cache, out[1], scores)
        assert cache.page_table[:, 0].min() >= first or first == 0
        # without the others the pages move to the front
        refs[:first] = 0
        Y.yoco_paged_compact(cache, refs, workspace=ws)
        out.append(torch.zeros(3, 6, d, dtype=t, device="cuda"))
        Y.yoco_paged_attn_decode_scored(q[:3], cache, out[2], scores)
        Y.yoco_workspace_status(ws)
        assert cache.page_table.max() < 9
        return [x.cpu() for x in out] + [cache.page_table.cpu(), refs[:9].cpu()]

    new = [torch.randn(190, 2, d, generator=g).to(t).cuda() for _ in range(3)]
    q = torch.randn(52, 6, d, generator=g).to(t).cuda()
    far, near = served(lead + 3), served(0)
    for a, b in zip(far, near):
        assert torch.equal(a, b)
    assert torch.equal(far[1], far[2]) and bool(far[0].abs().sum(-1).gt(0).all())


def test_copy_leaves_out_what_names_no_page(Y):
    k = torch.randn(6, 2, 16, 64, device="cuda")
    v = torch.randn(6, 2, 16, 64, device="cuda")
    cache = Y.PagedKV(k.clone(), v.clone(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    moves = torch.tensor([[900, 0, 0, 0], [0, 3, 5, 0], [-1, 2, 5, 0], [1, 6, 5, 0], [1, 4, 17, 0], [2, 5, 16, 0]], dtype=torch.int32)
    Y.yoco_paged_copy(cache, moves.cuda())
    k[3, :, :5], v[3, :, :5], k[5], v[5] = k[0, :, :5], v[0, :, :5], k[2], v[2]
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
    moves[0, 0] = -3
    Y.yoco_paged_copy(cache, moves.cuda())
    assert torch.equal(cache.k, k)


def test_rounds_captured_into_a_graph(Y):
    s = Pair(Y, 6, 40, 16, 8)
    s.resize([20, 30, 0, 0, 7, 0])
    lens = torch.tensor([20, 30, 0, 0, 7, 0], dtype=torch.int32).cuda()
    src, dst = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([2, 3], dtype=torch.int32).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y.yoco_paged_fork(s.cache, s.refs, src, dst, workspace=s.ws)
        Y.yoco_paged_resize(s.cache, s.refs, lens, moves=s.moves, workspace=s.ws)
    for new, a, b in (([25, 30, 50, 33, 0, 1], [0, 1], [2, 3]), ([0, 30, 0, -1, 2, 1], [3], [4]), ([-1, 31, 3, -1, 2, 70], [1], [0])):
        a, b = (a * 2)[:2], (b + [99])[:2]
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        src.copy_(torch.tensor(a, dtype=torch.int32))
        dst.copy_(torch.tensor(b, dtype=torch.int32))
        s.m.fork(a, b)
        assert s.m.resize(new)
        g.replay()
        s.after(Y.YOCO_ERR_INVALID_ARG if 99 in b else None)


def test_binding_refuses_what_it_cannot_marshal(Y):
    s = Pair(Y, 3, 20, 16, 4)
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(refs=s.refs[:19]), dict(refs=s.refs.cpu()), dict(refs=s.refs.long()), dict(new_lens=n[:2]), dict(new_lens=n.cpu()),
                dict(moves=s.moves[:3]), dict(moves=s.moves[:, :3].contiguous()), dict(workspace=s.ws.cpu())):
        with pytest.raises(ValueError):
            Y.yoco_paged_resize(s.cache, **{**dict(refs=s.refs, new_lens=n), **bad})
    with pytest.raises(ValueError):
        Y.yoco_paged_fork(s.cache, s.refs, n[:2], n)
    with pytest.raises(ValueError):
        Y.yoco_paged_compact(s.cache, s.refs, moves=s.moves[:10])
    with pytest.raises(Y.YocoError):
        Y.yoco_paged_fork(s.cache, s.refs, torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(Y.YocoError):
        Y.yoco_paged_resize(s.cache, s.refs, s.cache.seq_lens)
    with pytest.raises(Y.YocoError):
        Y.yoco_paged_resize(s.cache, s.refs, n, workspace=s.ws[:-1])
