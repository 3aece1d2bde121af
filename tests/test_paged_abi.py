"""CPU checks of the paged-cache calls: bad arguments are refused on the host before
anything is launched (no call below reaches a GPU)."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def Y():
    import gated_retention_shared_gb300 as Y
    return Y


def cache(Y, **kw):
    f = dict(k=0x10000, v=0x20000, page_table=0x30000, seq_lens=0x40000, B=3, Hkv=2, d=128, page_size=64, max_pages=40,
             num_pages=100, dtype=Y.YOCO_BF16, rope_base=0.0)
    f.update(kw)
    return Y._PagedKVC(*(f[n] for n, _ in Y._PagedKVC._fields_))


def decode(Y, c, Hq=4, scale=0.1, window=0, sinks=0, Q=FAKE, O=FAKE, ws=FAKE, n=1 << 40):
    return Y.lib.yoco_paged_attn_decode(Q, Hq, ctypes.byref(c), scale, window, sinks, O, ws, n, None)


def prefill(Y, c, Hq=4, rows=10, cu=FAKE, scale=0.1, window=0, sinks=0, Q=FAKE, O=FAKE, ws=FAKE, n=1 << 40):
    return Y.lib.yoco_paged_attn_prefill(Q, Hq, cu, rows, ctypes.byref(c), scale, window, sinks, O, ws, n, None)


def append(Y, c, k=FAKE, kr=256, kh=128, v=FAKE, vr=256, vh=128, q=None, qr=0, qh=0, qo=None, Hq=0, cu=FAKE, rows=10,
           ws=FAKE, n=256):
    return Y.lib.yoco_paged_append(k, kr, kh, v, vr, vh, q, qr, qh, qo, Hq, cu, rows, ctypes.byref(c), ws, n, None)


@pytest.mark.parametrize("field,value,status", [
    ("k", 0, 1), ("v", 0, 1), ("page_table", 0, 1), ("seq_lens", 0, 1), ("dtype", 7, 1), ("B", 0, 1), ("B", -1, 1),
    ("Hkv", 0, 1), ("max_pages", 0, 1), ("num_pages", 0, 1), ("d", 96, 2), ("d", 0, 2), ("page_size", 8, 2),
    ("page_size", 48, 2), ("page_size", 2048, 2), ("page_size", -64, 2), ("k", 0x10008, 1), ("v", 0x20004, 1),
    ("page_table", 0x30002, 1), ("seq_lens", 0x40001, 1), ("B", 4097, 2), ("max_pages", 1 << 25, 2),
    ("Hkv", 1 << 20, 2), ("rope_base", 1.0, 1), ("rope_base", -5.0, 1), ("rope_base", float("inf"), 1),
    ("rope_base", float("nan"), 1)])
def test_bad_cache_is_refused_by_every_call(Y, field, value, status):
    c = cache(Y, **{field: value})
    Hq = 4 if field != "Hkv" else max(1, 2 * value)
    assert decode(Y, c, Hq=Hq) == status
    assert prefill(Y, c, Hq=Hq) == status
    assert append(Y, c) == status
    assert Y.lib.yoco_last_error()
    assert Y.lib.yoco_paged_attn_workspace_size(Hq, 10, ctypes.byref(c)) == 0


def test_tiles_of_all_sequences_stay_below_2_30(Y):
    most = dict(B=4096, Hkv=16, page_size=128)
    assert prefill(Y, cache(Y, max_pages=1 << 14, **most), Hq=16, rows=0) == Y.YOCO_OK
    assert prefill(Y, cache(Y, max_pages=(1 << 14) + 1, **most), Hq=16, rows=0) == Y.YOCO_ERR_UNSUPPORTED


def test_calls_of_no_rows_take_null_tensors(Y):
    """What a binding hands over for an empty tensor."""
    assert prefill(Y, cache(Y), rows=0, Q=None, O=None) == Y.YOCO_OK
    assert prefill(Y, cache(Y), rows=0, Q=None, O=None, cu=None) == Y.YOCO_ERR_INVALID_ARG
    assert append(Y, cache(Y), k=None, v=None, rows=0) == Y.YOCO_OK
    assert append(Y, cache(Y), k=None, v=None, rows=1) == Y.YOCO_ERR_INVALID_ARG


def test_null_cache(Y):
    L = Y.lib
    assert L.yoco_paged_attn_decode(FAKE, 4, None, 0.1, 0, 0, FAKE, FAKE, 1 << 30, None) == Y.YOCO_ERR_INVALID_ARG
    assert L.yoco_paged_attn_prefill(FAKE, 4, FAKE, 1, None, 0.1, 0, 0, FAKE, FAKE, 1 << 30, None) == \
        Y.YOCO_ERR_INVALID_ARG
    assert L.yoco_paged_append(FAKE, 256, 128, FAKE, 256, 128, None, 0, 0, None, 0, FAKE, 1, None, FAKE, 256, None) == \
        Y.YOCO_ERR_INVALID_ARG
    assert L.yoco_paged_attn_workspace_size(4, 1, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=0), 2), (dict(Hq=5), 2), (dict(Hq=34), 2), (dict(Hq=-4), 2), (dict(Q=None), 1), (dict(O=None), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(Q=ctypes.c_void_p(0x10008)), 1),
    (dict(O=ctypes.c_void_p(0x10008)), 1), (dict(ws=None), 6), (dict(n=256), 6), (dict(ws=ctypes.c_void_p(0x10010)), 6)])
def test_bad_attention_arguments(Y, kw, status):
    c = cache(Y)
    assert decode(Y, c, **kw) == status
    assert prefill(Y, c, **kw) == status


def test_bad_prefill_rows(Y):
    c = cache(Y)
    assert prefill(Y, c, cu=None) == Y.YOCO_ERR_INVALID_ARG
    assert prefill(Y, c, cu=ctypes.c_void_p(0x10002)) == Y.YOCO_ERR_INVALID_ARG
    assert prefill(Y, c, rows=-1) == Y.YOCO_ERR_INVALID_ARG
    assert prefill(Y, c, rows=1 << 30) == Y.YOCO_ERR_UNSUPPORTED
    assert prefill(Y, c, rows=0) == Y.YOCO_OK  # nothing to do


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=None, v=None), 1), (dict(q=FAKE), 1), (dict(qo=FAKE), 1),
    (dict(q=FAKE, qo=FAKE, qr=512, qh=128, Hq=0), 1), (dict(rows=-1), 1), (dict(rows=(1 << 30) + 1), 2),
    (dict(q=FAKE, qo=ctypes.c_void_p(0x50000), qr=512, qh=128, Hq=8, rows=1 << 29), 2),
    (dict(cu=None, rows=4), 1), (dict(cu=ctypes.c_void_p(0x10001)), 1), (dict(k=ctypes.c_void_p(0x10008)), 1),
    (dict(v=ctypes.c_void_p(0x10008)), 1), (dict(kr=257), 1), (dict(kh=4), 1), (dict(vr=1), 1), (dict(vh=129), 1),
    (dict(q=FAKE, qo=ctypes.c_void_p(0x50008), qr=512, qh=128, Hq=4), 1),
    (dict(q=FAKE, qo=ctypes.c_void_p(0x50000), qr=511, qh=128, Hq=4), 1),
    (dict(q=FAKE, qo=FAKE, qr=1024, qh=128, Hq=4), 1), (dict(ws=None), 6), (dict(n=255), 6)])
def test_bad_append_arguments(Y, kw, status):
    assert append(Y, cache(Y), **kw) == status


def test_append_of_nothing(Y):
    assert append(Y, cache(Y), rows=0) == Y.YOCO_OK


def test_workspace_size_covers_every_call(Y):
    """One size serves decode and prefill, grows with the rows only where keys are split, and is
    small next to the cache."""
    c = cache(Y, B=64, Hkv=8, max_pages=2048, num_pages=4096)
    small = Y.lib.yoco_paged_attn_workspace_size(24, 64, ctypes.byref(c))
    large = Y.lib.yoco_paged_attn_workspace_size(24, 65536, ctypes.byref(c))
    assert 0 < small and 0 < large < 1 << 28
    assert Y.lib.yoco_paged_attn_workspace_size(25, 64, ctypes.byref(c)) == 0
    assert Y.lib.yoco_paged_attn_workspace_size(24, -1, ctypes.byref(c)) == 0


def test_python_binding_refuses_what_it_cannot_marshal(Y):
    import torch
    t = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError):  # not on a GPU
        Y.PagedKV(t, t, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
