"""GPU checks of a resize that comes upon counts of refs below what the tables say: what stays as it is,
and that the rest goes by the host's model, the same every time."""
import pytest
import torch

import test_gpu_paged_pool as Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Y():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import gated_retention_shared_gb300 as Y
    return Y


def lower(s, page, by=1):
    s.refs[page] -= by
    s.m.refs[page] -= by


def resize(s, new, stay, status):
    """The sequences `stay` are left as the model has them; everything else as documented."""
    fits = s.m.resize([-1 if b in stay else n for b, n in enumerate(new)])
    s.Y.yoco_paged_resize(s.cache, s.refs, torch.tensor(new, dtype=torch.int32).cuda(), moves=s.moves, workspace=s.ws)
    s.after(status)
    return fits


def owners(s):
    """How many sequences name each page."""
    held = [set(row[:s.m.held(n)]) for row, n in zip(s.cache.page_table.tolist(), s.cache.seq_lens.tolist())]
    return [sum(p in h for h in held) for p in range(len(s.m.refs))]


def test_more_growing_sequences_than_the_count(Y):
    for again in range(5):
        s = Pool.Pair(Y, 8, 40, 16, 8)
        s.resize([0, 20, 0, 0, 37, 0, 0, 0])
        s.fork([1, 1, 4], [0, 2, 5])  # 0, 1 and 2 share their pages, 4 and 5 theirs
        shared = s.m.table[1][1]
        lower(s, shared)  # counted 2, named 3 times
        before = owners(s)
        resize(s, [21, 25, 40, 70, 40, 41, 100, -1], {0, 1, 2}, Y.YOCO_ERR_INVALID_ARG)
        now = owners(s)
        assert now[shared] == before[shared] == 3 and s.refs[shared] == 2
        assert all(n <= 1 for p, n in enumerate(now) if before[p] == 0)  # what was handed out has one owner
        s.refs[shared] += 1  # put right, the next call serves them
        s.m.refs[shared] += 1
        s.resize([21, 25, 40, -1, -1, -1, -1, 16])


def test_a_page_that_is_counted_zero(Y):
    s = Pool.Pair(Y, 4, 20, 16, 8)
    s.resize([20, 33, 7, 0])
    page = s.m.table[1][2]
    lower(s, page)
    resize(s, [-1, 60, -1, -1], {1}, Y.YOCO_ERR_INVALID_ARG)
    assert s.cache.seq_lens.tolist() == [20, 33, 7, 0] and int(s.refs[page]) == 0


def test_low_counts_and_no_room(Y):
    s = Pool.Pair(Y, 5, 8, 16, 8)
    s.resize([20, 0, 0, 40, 0])
    s.fork([0, 0, 3], [1, 2, 4])
    lower(s, s.m.table[0][1])
    assert not resize(s, [25, 25, 25, 90, 90], {0, 1, 2}, Y.YOCO_ERR_CAPACITY)
    assert resize(s, [25, 25, 25, 41, 42], {0, 1, 2}, Y.YOCO_ERR_INVALID_ARG)


@pytest.mark.parametrize("B,each", [(40, 2), (1100, 5), (4096, 4)])
def test_many_low_counts(Y, B, each):
    """Groups of sequences that share their pages and all grow; every third group's page is counted too low."""
    want = None
    for again in range(3):
        s = Pool.Pair(Y, B, 4 * B, 16, 6, Hkv=1, dtype=torch.bfloat16)
        groups = B // each
        lens = [0] * B
        for g in range(groups):
            lens[g] = 17 + g % 15
        s.resize(lens)
        src = [g for g in range(groups) for _ in range(each - 1)]
        s.fork(src, list(range(groups, groups + len(src))))
        stay = set()
        for g in range(0, groups, 3):
            if each == 2:  # (a count of 1 is one sequence's)
                lower(s, s.m.table[g][1], 2)
            else:
                lower(s, s.m.table[g][1], 1 + g % (each - 2))
            stay |= {g} | {groups + i for i, a in enumerate(src) if a == g}
        if each == 2:  # pages counted 0 are free: nobody is given any here
            resize(s, [n + 1 if b in stay and n % 16 else -1 for b, n in enumerate(s.m.lens)], stay, Y.YOCO_ERR_INVALID_ARG)
        else:
            resize(s, [n + 1 + b % 30 if n else -1 for b, n in enumerate(s.m.lens)], stay, Y.YOCO_ERR_INVALID_ARG)
        got = (s.cache.page_table.clone(), s.refs.clone())
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
