"""CPU checks of the scored paged calls, the scaled rotary calls and the page calls: bad arguments are
refused on the host before anything is launched (no call below reaches a GPU)."""
import ctypes

import pytest

from test_paged_abi import FAKE, cache

F = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]  # never dereferenced


@pytest.fixture(scope="module")
def Y():
    import gated_retention_shared_gb300 as Y
    return Y


def rope_c(Y, **kw):
    f = dict(rotary_dim=0, layout=0, scaling=0, base=1e4, factor=1.0, original=4096.0, low=1.0, high=32.0, magnitude=1.0)
    f.update(kw)
    return Y._RopeC(*(f[n] for n, _ in Y._RopeC._fields_))


def rope(Y, r, x=F[0], xr=512, xh=128, out=F[1], orow=512, oh=128, rows=10, H=4, d=128, positions=F[2], pos0=0, dt=1):
    return Y.lib.yoco_rope_apply_scaled(x, xr, xh, out, orow, oh, rows, H, d, positions, pos0, None if r is None else ctypes.byref(r), dt, None)


def append(Y, r, c=None, **kw):
    c = c or cache(Y)
    return Y.lib.yoco_paged_append_rope(F[0], 256, 128, F[1], 256, 128, None, 0, 0, None, 0, F[2], kw.get("rows", 10), ctypes.byref(c),
                                        None if r is None else ctypes.byref(r), F[3], kw.get("n", 256), None)


inf, nan = float("inf"), float("nan")


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=8), 2), (dict(rotary_dim=-16), 2), (dict(rotary_dim=144), 2), (dict(rotary_dim=33), 2), (dict(layout=2), 1),
    (dict(layout=-1), 1), (dict(scaling=4), 1), (dict(scaling=-1), 1), (dict(base=1.0), 1), (dict(base=inf), 1), (dict(base=nan), 1),
    (dict(magnitude=0.0), 1), (dict(magnitude=-1.0), 1), (dict(magnitude=nan), 1), (dict(magnitude=inf), 1),
    (dict(scaling=1, factor=0.5), 1), (dict(scaling=2, factor=nan), 1), (dict(scaling=3, factor=inf), 1),
    (dict(scaling=3, original=0.0), 1), (dict(scaling=3, original=inf), 1), (dict(scaling=3, low=2.0, high=2.0), 1),
    (dict(scaling=3, low=3.0, high=2.0), 1), (dict(scaling=3, low=nan), 1), (dict(scaling=3, high=inf), 1)])
def test_bad_rotations_are_refused(Y, kw, status):
    assert rope(Y, rope_c(Y, **kw)) == status
    assert append(Y, rope_c(Y, **kw)) == status
    assert Y.lib.yoco_last_error()


def test_what_a_scaling_does_not_use_is_not_looked_at(Y):
    assert rope(Y, rope_c(Y, factor=nan, original=-1.0, low=5.0, high=1.0), rows=0) == Y.YOCO_OK
    assert rope(Y, rope_c(Y, scaling=1, factor=2.0, original=-1.0), rows=0) == Y.YOCO_OK


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(x=ctypes.c_void_p(0x10008)), 1), (dict(out=ctypes.c_void_p(0x10008)), 1),
    (dict(xr=513), 1), (dict(xh=4), 1), (dict(orow=1), 1), (dict(oh=132), 1), (dict(rows=-1), 1), (dict(H=0), 1), (dict(d=96), 2),
    (dict(dt=2), 1), (dict(rows=1 << 30), 2), (dict(positions=ctypes.c_void_p(0x30002)), 1), (dict(out=F[0], orow=1024), 1),
    (dict(positions=None, pos0=(1 << 31) - 9), 1), (dict(positions=None, pos0=-(1 << 31)), 1), (dict(positions=None, pos0=1 << 62), 1),
    (dict(positions=None, pos0=-(1 << 63)), 1)])
def test_bad_rope_arguments(Y, kw, status):
    assert rope(Y, rope_c(Y), **kw) == status


@pytest.mark.parametrize("kw", [dict(orow=0), dict(oh=0), dict(out=F[0], xr=0, orow=0), dict(out=F[0], xh=0, oh=0)])
def test_rows_or_heads_that_come_out_in_one_place_are_refused(Y, kw):
    assert rope(Y, rope_c(Y), **kw) == Y.YOCO_ERR_INVALID_ARG
    assert rope(Y, rope_c(Y), **kw, rows=0) == (Y.YOCO_ERR_INVALID_ARG if "oh" in kw else Y.YOCO_OK)


def test_null_and_empty_rope_calls(Y):
    assert rope(Y, None) == Y.YOCO_ERR_INVALID_ARG
    assert append(Y, None) == Y.YOCO_ERR_INVALID_ARG
    assert rope(Y, rope_c(Y), rows=0, x=None, out=None) == Y.YOCO_OK
    assert append(Y, rope_c(Y), rows=0) == Y.YOCO_OK
    assert append(Y, rope_c(Y), c=cache(Y, rope_base=1e4)) == Y.YOCO_ERR_INVALID_ARG
    assert append(Y, rope_c(Y, rotary_dim=128), c=cache(Y, d=64)) == Y.YOCO_ERR_UNSUPPORTED
    assert append(Y, rope_c(Y), n=255) == Y.YOCO_ERR_WORKSPACE


def scores_c(Y, softcap=0.0, slopes=None, prefix=None, doc=None):
    return Y._PagedScoresC(softcap, slopes, prefix, doc)


def attn(Y, s, c=None, scale=0.1, ws=FAKE, n=1 << 40, Q=F[0], O=F[1], cu=F[2], Hq=4, rows=10, window=0, sinks=0):
    c = c or cache(Y)
    s = None if s is None else ctypes.byref(s)
    return (Y.lib.yoco_paged_attn_prefill_scored(Q, Hq, cu, rows, ctypes.byref(c), s, scale, window, sinks, O, ws, n, None),
            Y.lib.yoco_paged_attn_decode_scored(Q, Hq, ctypes.byref(c), s, scale, window, sinks, O, ws, n, None))


@pytest.mark.parametrize("kw", [dict(softcap=-1.0), dict(softcap=nan), dict(softcap=inf), dict(softcap=1e-30), dict(softcap=1e30),
                                dict(slopes=0x10001), dict(prefix=0x10002), dict(doc=0x10003)])
def test_bad_scores_are_refused(Y, kw):
    assert attn(Y, scores_c(Y, **kw)) == (1, 1)
    assert Y.lib.yoco_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=nan), 1), (dict(Q=None), 1), (dict(O=None), 1), (dict(Hq=5), 2),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(Q=ctypes.c_void_p(0x10008)), 1), (dict(ws=None), 6), (dict(n=256), 6),
    (dict(scale=1e30), 1)])
def test_bad_scored_arguments(Y, kw, status):
    assert attn(Y, scores_c(Y, softcap=5.0), **kw) == (status, status)


def test_null_scores_and_cache(Y):
    assert attn(Y, None) == (1, 1)
    assert Y.lib.yoco_paged_attn_decode_scored(F[0], 4, None, ctypes.byref(scores_c(Y)), 0.1, 0, 0, F[1], FAKE, 1 << 30, None) == 1
    assert attn(Y, scores_c(Y), cu=None)[0] == 1


@pytest.mark.parametrize("field,value,status", [
    ("k", 0, 1), ("page_table", 0, 1), ("B", 0, 1), ("d", 96, 2), ("page_size", 48, 2), ("B", 4097, 2), ("num_pages", 0, 1),
    ("max_pages", 1 << 25, 2)])
def test_bad_cache_is_refused_by_every_page_call(Y, field, value, status):
    c = ctypes.byref(cache(Y, **{field: value}))
    L = Y.lib
    assert L.yoco_paged_pool_workspace_size(c) == 0
    assert L.yoco_paged_resize(c, F[0], F[1], None, FAKE, 1 << 40, None) == status
    assert L.yoco_paged_fork(c, F[0], F[1], F[2], 1, FAKE, 1 << 40, None) == status
    assert L.yoco_paged_compact(c, F[0], None, FAKE, 1 << 40, None) == status
    assert L.yoco_paged_copy(c, F[0], 1, None) == status


def test_bad_page_arguments(Y):
    L, kv = Y.lib, cache(Y)
    c = ctypes.byref(kv)
    odd, ws, n = ctypes.c_void_p(0x10008), FAKE, L.yoco_paged_pool_workspace_size(c)
    assert n > 0
    INVALID, WORKSPACE = Y.YOCO_ERR_INVALID_ARG, Y.YOCO_ERR_WORKSPACE
    assert L.yoco_paged_resize(None, F[0], F[1], None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, None, F[1], None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, ctypes.c_void_p(0x10002), F[1], None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, F[0], None, None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, F[0], ctypes.c_void_p(0x10001), None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, F[0], ctypes.c_void_p(kv.seq_lens), None, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, F[0], F[1], odd, ws, n, None) == INVALID
    assert L.yoco_paged_resize(c, F[0], F[1], None, None, n, None) == WORKSPACE
    assert L.yoco_paged_resize(c, F[0], F[1], None, odd, n, None) == WORKSPACE
    assert L.yoco_paged_resize(c, F[0], F[1], None, ws, n - 1, None) == WORKSPACE
    assert L.yoco_paged_fork(c, F[0], None, F[1], 1, ws, n, None) == INVALID
    assert L.yoco_paged_fork(c, F[0], F[1], None, 1, ws, n, None) == INVALID
    assert L.yoco_paged_fork(c, F[0], F[1], F[2], -1, ws, n, None) == INVALID
    assert L.yoco_paged_fork(c, F[0], F[1], F[2], 4, ws, n, None) == INVALID  # more than there are sequences
    assert L.yoco_paged_fork(c, F[0], None, None, 0, ws, n, None) == Y.YOCO_OK
    assert L.yoco_paged_compact(c, None, None, ws, n, None) == INVALID
    assert L.yoco_paged_compact(c, F[0], odd, ws, n, None) == INVALID
    assert L.yoco_paged_compact(c, F[0], None, ws, n - 1, None) == WORKSPACE
    assert L.yoco_paged_copy(c, None, 1, None) == INVALID
    assert L.yoco_paged_copy(c, odd, 1, None) == INVALID
    assert L.yoco_paged_copy(c, F[0], -1, None) == INVALID
    assert L.yoco_paged_copy(c, F[0], 0, None) == Y.YOCO_OK


def test_injected_launch_failures_reach_every_new_call(Y):
    """After the checks and before any launch, so these reach no GPU either."""
    L, c = Y.lib, ctypes.byref(cache(Y))
    n = 1 << 40
    calls = [lambda: rope(Y, rope_c(Y)), lambda: append(Y, rope_c(Y)), lambda: attn(Y, scores_c(Y))[0],
             lambda: L.yoco_paged_attn_decode_scored(F[0], 4, c, ctypes.byref(scores_c(Y)), 0.1, 0, 0, F[1], FAKE, n, None),
             lambda: L.yoco_paged_resize(c, F[0], F[1], None, FAKE, n, None), lambda: L.yoco_paged_fork(c, F[0], F[1], F[2], 1, FAKE, n, None),
             lambda: L.yoco_paged_compact(c, F[0], None, FAKE, n, None), lambda: L.yoco_paged_copy(c, F[0], 1, None)]
    try:
        for call in calls:
            assert L.yoco_test_hook(Y.YOCO_HOOK_FAIL_NEXT_CALLS, 2) == Y.YOCO_OK
            assert call() == Y.YOCO_ERR_CUDA
    finally:
        L.yoco_test_hook(Y.YOCO_HOOK_FAIL_NEXT_CALLS, 0)


def test_python_side_refusals(Y):
    for bad in (dict(layout="quarters"), dict(scaling="log"), dict(rotary_dim=0), dict(rotary_dim=-16)):
        with pytest.raises(ValueError):
            Y.Rope(**bad)
    import torch
    with pytest.raises(ValueError):  # not on a GPU
        Y.PagedScores(slopes=torch.zeros(4))
    with pytest.raises(ValueError):
        Y.yoco_rope_apply_scaled(torch.zeros(2, 3, 64), Y.Rope())
