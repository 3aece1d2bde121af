"""Python binding of libyoco (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of the method: it reads shapes and device pointers off torch
tensors, passes them with the current CUDA stream through ctypes, and raises
on a non-OK status.  All computation runs in the CUDA kernels of
``_build/libyoco.so``; there is no fallback.  If the library is missing the
import fails with a message saying how to build it.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# YOCO_LIB_PATH selects another build of the same library (the debug-checks build
# in _build_debug/, for its tests); the default is the release build
LIB_PATH = os.environ.get("YOCO_LIB_PATH") or os.path.join(_HERE, "_build", "libyoco.so")

YOCO_OK, YOCO_ERR_INVALID_ARG, YOCO_ERR_UNSUPPORTED, YOCO_ERR_CAPACITY, YOCO_ERR_CUDA, YOCO_ERR_TIMEOUT, \
    YOCO_ERR_WORKSPACE = range(7)
YOCO_F32, YOCO_BF16 = 0, 1


class YocoError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


class _KVCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len_dev", ctypes.c_void_p),
                ("len_host", ctypes.c_int64), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("capacity", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("rope_base", ctypes.c_float)]


class _SwaRingC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("window", ctypes.c_int32), ("pos", ctypes.c_int64), ("dtype", ctypes.c_int)]


class _PagedKVC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("rope_base", ctypes.c_float)]


class _RopeC(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_float), ("factor", ctypes.c_float), ("original", ctypes.c_float),
                ("low", ctypes.c_float), ("high", ctypes.c_float), ("magnitude", ctypes.c_float)]


class _PagedScoresC(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p),
                ("doc_first", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libyoco.so not found at {LIB_PATH}; build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    cp = ctypes.POINTER(_KVCacheC)
    rp = ctypes.POINTER(_SwaRingC)
    pp = ctypes.POINTER(_PagedKVC)
    op = ctypes.POINTER(_RopeC)
    cs = ctypes.POINTER(_PagedScoresC)
    sigs = {
        "yoco_gret_prefill_chunkwise": (i, [vp, vp, vp, vp, f, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]),
        "yoco_gret_prefill_workspace_size": (sz, [i, i, i, i, i, i, i]),
        "yoco_gret_decode_step": (i, [vp, vp, vp, vp, f, vp, vp, i, i, i, i, i, i, vp]),
        "yoco_shared_kv_project_append": (i, [vp, vp, f, vp, vp, i, i, cp, vp, sz, vp]),
        "yoco_shared_kv_workspace_size": (sz, [i, i, i, cp]),
        "yoco_cross_attn_prefill": (i, [vp, i, i, i64, cp, f, vp, vp, sz, vp]),
        "yoco_cross_attn_decode": (i, [vp, i, cp, f, i, vp, vp, sz, vp]),
        "yoco_cross_attn_workspace_size": (sz, [i, i, i, cp, i]),
        "yoco_cross_attn_decode_noalloc": (i, [vp, i, cp, f, i, vp, vp]),
        "yoco_status_string": (ctypes.c_char_p, [i]),
        "yoco_last_error": (ctypes.c_char_p, []),
        "yoco_version": (i, []),
        "yoco_launch_count": (ctypes.c_uint64, []),
        "yoco_workspace_status": (i, [vp, i, vp]),
        "yoco_selftest_wait_timeout": (i, [vp, ctypes.c_uint64, vp]),
        "yoco_swa_prefill": (i, [vp, vp, vp, i, i, f, vp, rp, vp, sz, vp]),
        "yoco_swa_decode": (i, [vp, vp, vp, i, f, vp, rp, vp, sz, vp]),
        "yoco_swa_workspace_size": (sz, [i, i, rp]),
        "yoco_gret_group_norm_gate": (i, [vp, vp, vp, vp, f, vp, i, i, i, i, i, vp]),
        "yoco_gret_decode_step_gn_gate": (i, [vp, vp, vp, vp, f, vp, vp, vp, vp, f, vp, i, i, i, i, i, vp]),
        "yoco_rope_apply": (i, [vp, i, i, i, i, i64, f, i, vp]),
        "yoco_gret_qkvg_project": (i, [vp, vp, i, i, i, i, i, i64, f, vp, vp, vp, vp, vp, sz, vp]),
        "yoco_gret_qkvg_workspace_size": (sz, [i, i, i, i, f]),
        "yoco_cross_attn_decode_noalloc_status": (i, [i, vp]),
        "yoco_test_hook": (i, [i, i64]),
        "yoco_gret_prefill_chunkwise_gn_gate": (i, [vp, vp, vp, vp, f, vp, vp, vp, f, vp, vp, i, i, i, i, i, i, vp, sz,
                                                    vp]),
        "yoco_selftest_occupy_sms": (i, [i, ctypes.c_uint64, vp]),
        "yoco_paged_append": (i, [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i, vp, i, pp, vp, sz, vp]),
        "yoco_paged_attn_prefill": (i, [vp, i, vp, i, pp, f, i, i, vp, vp, sz, vp]),
        "yoco_paged_attn_decode": (i, [vp, i, pp, f, i, i, vp, vp, sz, vp]),
        "yoco_paged_attn_workspace_size": (sz, [i, i, pp]),
        "yoco_rope_apply_scaled": (i, [vp, i64, i64, vp, i64, i64, i, i, i, vp, i64, op, i, vp]),
        "yoco_paged_append_rope": (i, [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i, vp, i, pp, op, vp, sz, vp]),
        "yoco_paged_attn_prefill_scored": (i, [vp, i, vp, i, pp, cs, f, i, i, vp, vp, sz, vp]),
        "yoco_paged_attn_decode_scored": (i, [vp, i, pp, cs, f, i, i, vp, vp, sz, vp]),
        "yoco_paged_resize": (i, [pp, vp, vp, vp, vp, sz, vp]),
        "yoco_paged_fork": (i, [pp, vp, vp, vp, i, vp, sz, vp]),
        "yoco_paged_compact": (i, [pp, vp, vp, vp, sz, vp]),
        "yoco_paged_copy": (i, [pp, vp, i, vp]),
        "yoco_paged_pool_workspace_size": (sz, [pp]),
        "yoco_debug_checks": (i, [i, ctypes.POINTER(ctypes.c_uint32)]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()
EXPORTED = ("yoco_gret_prefill_chunkwise", "yoco_gret_prefill_workspace_size", "yoco_gret_decode_step",
            "yoco_shared_kv_project_append", "yoco_shared_kv_workspace_size", "yoco_cross_attn_prefill",
            "yoco_cross_attn_decode", "yoco_cross_attn_workspace_size", "yoco_status_string",
            "yoco_last_error", "yoco_version", "yoco_launch_count",
            "yoco_workspace_status", "yoco_cross_attn_decode_noalloc", "yoco_selftest_wait_timeout",
            "yoco_swa_prefill", "yoco_swa_decode", "yoco_swa_workspace_size", "yoco_gret_group_norm_gate",
            "yoco_rope_apply", "yoco_gret_qkvg_project", "yoco_gret_qkvg_workspace_size",
            "yoco_gret_decode_step_gn_gate", "yoco_cross_attn_decode_noalloc_status", "yoco_test_hook",
            "yoco_selftest_occupy_sms", "yoco_gret_prefill_chunkwise_gn_gate", "yoco_debug_checks", "yoco_paged_append",
            "yoco_paged_attn_prefill", "yoco_paged_attn_decode", "yoco_paged_attn_workspace_size",
            "yoco_rope_apply_scaled", "yoco_paged_append_rope", "yoco_paged_attn_prefill_scored",
            "yoco_paged_attn_decode_scored", "yoco_paged_resize", "yoco_paged_fork", "yoco_paged_compact",
            "yoco_paged_copy", "yoco_paged_pool_workspace_size")
YOCO_HOOK_FAIL_NEXT_CALLS, YOCO_HOOK_GRET_SEG0_DELAY_NS, YOCO_HOOK_GRET_SEGMENTS = 1, 2, 3


def _check(status: int, where: str):
    if status != YOCO_OK:
        detail = lib.yoco_last_error().decode() or lib.yoco_status_string(status).decode()
        raise YocoError(status, where, detail)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return YOCO_F32
    if t.dtype == torch.bfloat16:
        return YOCO_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _workspace(nbytes: int, device, workspace, stream):
    if nbytes == 0:
        return workspace
    if workspace is None:
        workspace = _scratch(nbytes, device, stream)
    return workspace


def _scratch(nbytes: int, device, stream):
    """A workspace of the binding's own from the pool of the stream that will use it.  What the
    current stream's pool hands out may be memory that is free to that stream's later work only:
    work queued there before may still write it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # another library's
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ gRet

def yoco_gret_prefill_workspace_size(B, N, H, dk, dv, chunk, dtype) -> int:
    return lib.yoco_gret_prefill_workspace_size(B, N, H, dk, dv, chunk, dtype)


def yoco_gret_prefill_chunkwise(q, k, v, gate_logits, tau, o, state, chunk=0, workspace=None, stream=None):
    """q, k [B,N,H,dk]; v, o [B,N,H,dv]; gate_logits [B,N,H] fp32; state [B,H,dk,dv] fp32 (in/out)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (gate_logits, "gate_logits"), (o, "o"), (state, "state")):
        _need(t, n)
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    ws_n = lib.yoco_gret_prefill_workspace_size(B, N, H, dk, dv, chunk, dt)
    ws = _workspace(ws_n, q.device, workspace, stream)
    st = lib.yoco_gret_prefill_chunkwise(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_logits), float(tau), _ptr(o),
                                         _ptr(state), B, N, H, dk, dv, chunk, dt, _dt(o), _ptr(ws),
                                         0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_gret_prefill_chunkwise")


def yoco_gret_prefill_chunkwise_gn_gate(q, k, v, gate_logits, tau, gate, z, state, eps=1e-5, gn_weight=None,
                                        gn_bias=None, workspace=None, stream=None):
    """z = swish(gate) * GroupNorm_h(chunkwise gRet output); q, k, v, gate, z [B,N,H,d];
    gate_logits [B,N,H] fp32; state [B,H,d,d] fp32 (in/out); gn_weight, gn_bias fp32 [H*d] or None."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (gate_logits, "gate_logits"), (gate, "gate"), (z, "z"),
                 (state, "state")):
        _need(t, n)
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    for t, n in ((gn_weight, "gn_weight"), (gn_bias, "gn_bias")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != H * dv):
            raise ValueError(f"{n} must be fp32 with H * d elements")
    ws_n = lib.yoco_gret_prefill_workspace_size(B, N, H, dk, dv, 0, dt)
    ws = _workspace(ws_n, q.device, workspace, stream)
    st = lib.yoco_gret_prefill_chunkwise_gn_gate(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_logits), float(tau), _ptr(gate),
                                                 _ptr(gn_weight), _ptr(gn_bias), float(eps), _ptr(z), _ptr(state), B, N,
                                                 H, dk, dv, dt, _ptr(ws),
                                                 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_gret_prefill_chunkwise_gn_gate")


def yoco_workspace_status(workspace, clear=True, stream=None):
    """Wait for the stream and raise YocoError(YOCO_ERR_TIMEOUT) if a kernel
    that used `workspace` gave up a bounded on-device wait."""
    _check(lib.yoco_workspace_status(_ptr(workspace), int(clear), _stream(stream)), "yoco_workspace_status")


def yoco_gret_decode_step(q, k, v, gate_logits, tau, state, o, stream=None):
    """q, k [B,H,dk]; v, o [B,H,dv]; gate_logits [B,H] fp32; state [B,H,dk,dv] fp32 (in/out)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (gate_logits, "gate_logits"), (o, "o"), (state, "state")):
        _need(t, n)
    B, H, dk = q.shape
    dv = v.shape[-1]
    st = lib.yoco_gret_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_logits), float(tau), _ptr(state),
                                   _ptr(o), B, H, dk, dv, _dt(q), _dt(o), _stream(stream))
    _check(st, "yoco_gret_decode_step")


def yoco_gret_decode_step_gn_gate(q, k, v, gate_logits, tau, state, gate, z, eps=1e-5, gn_weight=None, gn_bias=None,
                                  stream=None):
    """One recurrent step and, fused, z = swish(gate) * GroupNorm_h(o) for that token.
    q, k [B,H,dk]; v, gate, z [B,H,dv] (one dtype); gate_logits [B,H] fp32; state
    [B,H,dk,dv] fp32 (in/out); gn_weight, gn_bias fp32 [H * dv] or None."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (gate_logits, "gate_logits"), (state, "state"), (gate, "gate"),
                 (z, "z")):
        _need(t, n)
    B, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((gn_weight, "gn_weight"), (gn_bias, "gn_bias")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != H * dv):
            raise ValueError(f"{n} must be fp32 with H * dv elements")
    st = lib.yoco_gret_decode_step_gn_gate(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_logits), float(tau), _ptr(state),
                                           _ptr(gate), _ptr(gn_weight), _ptr(gn_bias), float(eps), _ptr(z), B, H, dk,
                                           dv, _dt(q), _stream(stream))
    _check(st, "yoco_gret_decode_step_gn_gate")


# ------------------------------------------------------------- shared KV

class KVCache:
    """Caller-side holder of the shared K^/V^ cache: two [B, Hkv, capacity, d]
    tensors, the device length pair and the C descriptor that points at them."""

    def __init__(self, B, Hkv, d, capacity, dtype=torch.bfloat16, device="cuda", k=None, v=None, rope_base=0.0):
        self.k = k if k is not None else torch.zeros(B, Hkv, capacity, d, dtype=dtype, device=device)
        self.v = v if v is not None else torch.zeros(B, Hkv, capacity, d, dtype=dtype, device=device)
        self.len_dev = torch.zeros(2, dtype=torch.int32, device=self.k.device)
        self.c = _KVCacheC(self.k.data_ptr(), self.v.data_ptr(), self.len_dev.data_ptr(), 0, B, Hkv, d,
                           capacity, _dt(self.k), float(rope_base))

    @property
    def length(self) -> int:
        return int(self.c.len_host)

    def set_length(self, n: int):
        """Declare the first n slots filled (e.g. after writing k/v directly)."""
        self.c.len_host = n
        self.len_dev[0] = n

    @staticmethod
    def nbytes(B, Hkv, d, capacity, elem_bytes=2) -> int:
        return 2 * B * Hkv * capacity * d * elem_bytes


def yoco_shared_kv_project_append(M, Wk, Wv, cache: KVCache, eps=1e-6, rms_w=None, workspace=None, stream=None):
    """M [B, T, dm]; Wk, Wv [dm, Hkv*d]; appends T slots to `cache`."""
    for t, n in ((M, "M"), (Wk, "Wk"), (Wv, "Wv")):
        _need(t, n)
    B, T, dm = M.shape
    ws_n = lib.yoco_shared_kv_workspace_size(B, T, dm, ctypes.byref(cache.c))
    ws = _workspace(ws_n, M.device, workspace, stream)
    st = lib.yoco_shared_kv_project_append(_ptr(M), _ptr(rms_w), float(eps), _ptr(Wk), _ptr(Wv), T, dm,
                                           ctypes.byref(cache.c), _ptr(ws),
                                           0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_shared_kv_project_append")


# -------------------------------------------------------- cross attention

def yoco_cross_attn_decode_noalloc(Q, cache: KVCache, O, scale=None, num_splits=0, stream=None):
    """Decode attention without a workspace: the split partials go to scratch
    built into the library, for callers that cannot allocate device memory.
    Calls on one device share that scratch, so do not overlap them."""
    _need(Q, "Q")
    _need(O, "O")
    B, Hq, d = Q.shape
    scale = d ** -0.5 if scale is None else scale
    st = lib.yoco_cross_attn_decode_noalloc(_ptr(Q), Hq, ctypes.byref(cache.c), float(scale), num_splits, _ptr(O),
                                            _stream(stream))
    _check(st, "yoco_cross_attn_decode_noalloc")


def yoco_cross_attn_workspace_size(B, Hq, T, cache: KVCache, num_splits=0) -> int:
    return lib.yoco_cross_attn_workspace_size(B, Hq, T, ctypes.byref(cache.c), num_splits)


def yoco_cross_attn_prefill(Q, cache: KVCache, p0, O, scale=None, workspace=None, stream=None):
    """Q, O [B, T, Hq, d]; rows at positions p0..p0+T-1."""
    _need(Q, "Q")
    _need(O, "O")
    B, T, Hq, d = Q.shape
    scale = d ** -0.5 if scale is None else scale
    ws_n = lib.yoco_cross_attn_workspace_size(B, Hq, T, ctypes.byref(cache.c), 0)
    ws = _workspace(ws_n, Q.device, workspace, stream)
    st = lib.yoco_cross_attn_prefill(_ptr(Q), Hq, T, int(p0), ctypes.byref(cache.c), float(scale), _ptr(O), _ptr(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_cross_attn_prefill")


def yoco_cross_attn_decode(Q, cache: KVCache, O, scale=None, num_splits=0, workspace=None, stream=None):
    """Q, O [B, Hq, d]; the query sits at position len - 1."""
    _need(Q, "Q")
    _need(O, "O")
    B, Hq, d = Q.shape
    scale = d ** -0.5 if scale is None else scale
    ws_n = lib.yoco_cross_attn_workspace_size(B, Hq, 1, ctypes.byref(cache.c), num_splits)
    ws = _workspace(ws_n, Q.device, workspace, stream)
    st = lib.yoco_cross_attn_decode(_ptr(Q), Hq, ctypes.byref(cache.c), float(scale), num_splits, _ptr(O), _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_cross_attn_decode")


# ----------------------------------------------- sliding-window self-decoder

class SwaRing:
    """Caller-side ring cache of one sliding-window layer: k, v [B, Hkv, window, d]
    (token at position p in slot p % window) and the C descriptor; `pos` counts
    the tokens seen."""

    def __init__(self, B, Hkv, d, window, dtype=torch.bfloat16, device="cuda"):
        self.k = torch.zeros(B, Hkv, window, d, dtype=dtype, device=device)
        self.v = torch.zeros(B, Hkv, window, d, dtype=dtype, device=device)
        self.c = _SwaRingC(self.k.data_ptr(), self.v.data_ptr(), B, Hkv, d, window, 0, _dt(self.k))

    @property
    def pos(self) -> int:
        return int(self.c.pos)


def yoco_swa_prefill(q, k, v, ring: SwaRing, o, scale=None, workspace=None, stream=None):
    """q, o [B, N, Hq, d]; k, v [B, N, Hkv, d]; starts the sequence held in `ring`."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    B, N, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    ws = _workspace(max(256, lib.yoco_swa_workspace_size(B, Hq, ctypes.byref(ring.c))), q.device, workspace, stream)
    st = lib.yoco_swa_prefill(_ptr(q), _ptr(k), _ptr(v), Hq, N, float(scale), _ptr(o), ctypes.byref(ring.c),
                              _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_swa_prefill")


def yoco_swa_decode(q, k, v, ring: SwaRing, o, scale=None, workspace=None, stream=None):
    """q, o [B, Hq, d]; k, v [B, Hkv, d] of the new token."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    B, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    ws = _workspace(max(256, lib.yoco_swa_workspace_size(B, Hq, ctypes.byref(ring.c))), q.device, workspace, stream)
    st = lib.yoco_swa_decode(_ptr(q), _ptr(k), _ptr(v), Hq, float(scale), _ptr(o), ctypes.byref(ring.c), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "yoco_swa_decode")


def yoco_gret_group_norm_gate(o, gate, z, eps=1e-5, gn_weight=None, gn_bias=None, stream=None):
    """z = swish(gate) * GroupNorm_h(o); o, gate, z [B, N, H, d] (or [B, H, d] for a decode step);
    gn_weight, gn_bias fp32 [H * d] or None.  z may be o."""
    for t, n in ((o, "o"), (gate, "gate"), (z, "z")):
        _need(t, n)
    if o.dim() == 3:
        B, H, d = o.shape
        N = 1
    else:
        B, N, H, d = o.shape
    for t, n in ((gn_weight, "gn_weight"), (gn_bias, "gn_bias")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != H * d):
            raise ValueError(f"{n} must be fp32 with H * d elements")
    st = lib.yoco_gret_group_norm_gate(_ptr(o), _ptr(gate), _ptr(gn_weight), _ptr(gn_bias), float(eps), _ptr(z), B, N,
                                       H, d, _dt(o), _stream(stream))
    _check(st, "yoco_gret_group_norm_gate")


# ------------------------------------------------- rotary position encoding

def yoco_rope_apply(x, base, pos0=0, stream=None):
    """Rotary encoding of x [B, N, H, d] (token-major q or k) in place: row n at position pos0 + n."""
    _need(x, "x")
    B, N, H, d = x.shape
    st = lib.yoco_rope_apply(_ptr(x), B, N, H, d, int(pos0), float(base), _dt(x), _stream(stream))
    _check(st, "yoco_rope_apply")


class Rope:
    """A rotary encoding other than pairs of the whole head at one base: `rotary_dim` channels of each
    head (None: all), in "pairs" (2i, 2i+1) or "halves" (i, i + r/2), frequencies unscaled ("none"),
    "linear", "ntk" or "by_parts" (yoco.h has the formulas; its ramp is over turns), turned channels times `magnitude`."""
    LAYOUTS = {"pairs": 0, "halves": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}

    def __init__(self, rotary_dim=None, layout="pairs", base=1e4, scaling="none", factor=1.0, original=8192.0, low=1.0,
                 high=32.0, magnitude=1.0):
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise ValueError(f"layout is one of {list(self.LAYOUTS)}, scaling one of {list(self.SCALINGS)}")
        if rotary_dim is not None and rotary_dim <= 0:
            raise ValueError("rotary_dim must be positive")
        self.c = _RopeC(rotary_dim or 0, self.LAYOUTS[layout], self.SCALINGS[scaling], base, factor, original, low, high,
                        magnitude)
        self.ref = ctypes.byref(self.c)


def _rows_heads(t, name, like=None):
    """Pointer and strides of a [rows, heads, d] tensor with adjacent channels."""
    shape, stride = t.shape, t.stride()
    if not t.is_cuda or len(shape) != 3 or (stride[2] != 1 and shape[2] != 1):
        raise ValueError(f"{name} must be a CUDA tensor [rows, heads, d] with adjacent channels")
    if like is not None and (shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must have x's shape, dtype and device")
    # (the stride of an axis of one element means nothing, and may be anything)
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * shape[2], stride[1] if shape[1] > 1 else shape[2]


def yoco_rope_apply_scaled(x, rope: Rope, out=None, positions=None, pos0=0, stream=None):
    """x [rows, H, d] with any strides that are multiples of 16 bytes, turned into out (None: in
    place), row i at positions[i] (int32 [rows]) or, without them, at pos0 + i."""
    xp = _rows_heads(x, "x")
    op = xp if out is None else _rows_heads(out, "out", x)
    rows, H, d = x.shape
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != (rows,) or
                                  positions.device != x.device or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 [rows] on x's device")
    if not -2**31 <= pos0 <= 2**31:
        raise ValueError("pos0 is beyond 2^31")
    _device_call(lib.yoco_rope_apply_scaled, "yoco_rope_apply_scaled", x.get_device(), stream, *xp, *op, rows, H, d,
                 None if positions is None else positions.data_ptr(), pos0, rope.ref, _dt(x))


def yoco_gret_qkvg_project(X, W, H, q, k, v, gate_logits, rope_base=0.0, pos0=0, workspace=None, stream=None):
    """X [B, N, dm] bf16; W [dm, 3 H d + H] bf16 (W_Q | W_K | W_V | W_gamma); writes q, k, v
    [B, N, H, d] bf16 and gate_logits [B, N, H] fp32."""
    for t, n in ((X, "X"), (W, "W"), (q, "q"), (k, "k"), (v, "v"), (gate_logits, "gate_logits")):
        _need(t, n)
    B, N, dm = X.shape
    d = q.shape[-1]
    ws_n = lib.yoco_gret_qkvg_workspace_size(B, N, H, d, float(rope_base))
    ws = _workspace(ws_n, X.device, workspace, stream)
    st = lib.yoco_gret_qkvg_project(_ptr(X), _ptr(W), B, N, dm, H, d, int(pos0), float(rope_base), _ptr(q), _ptr(k),
                                    _ptr(v), _ptr(gate_logits), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream))
    _check(st, "yoco_gret_qkvg_project")


# ------------------------------------- many sequences on pages of one cache

class PagedKV:
    """Caller-side holder of a paged cache: k, v [num_pages, Hkv, page_size, d],
    page_table int32 [B, max_pages] and seq_lens int32 [B] on the device, and the C
    descriptor that points at them.  The caller hands out pages and advances
    seq_lens (to the lengths with a call's new rows) before the call."""

    def __init__(self, k, v, page_table, seq_lens, rope_base=0.0):
        for t, n in ((k, "k"), (v, "v"), (page_table, "page_table"), (seq_lens, "seq_lens")):
            _need(t, n)
            if t.device != k.device:
                raise ValueError(f"{n} is on {t.device}, k on {k.device}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be [num_pages, Hkv, page_size, d] of one dtype")
        if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
            raise TypeError("page_table and seq_lens must be int32")
        if page_table.dim() != 2 or seq_lens.shape != page_table.shape[:1]:
            raise ValueError("page_table must be [B, max_pages] and seq_lens [B]")
        self.k, self.v, self.page_table, self.seq_lens = k, v, page_table, seq_lens
        num_pages, Hkv, page_size, d = k.shape
        B, max_pages = page_table.shape
        self.c = _PagedKVC(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), B, Hkv, d, page_size,
                           max_pages, num_pages, _dt(k), float(rope_base))
        self.ref = ctypes.byref(self.c)
        # what every call's checks ask for, in plain attributes: a call of one token per sequence
        # takes the GPU a few microseconds, so the binding must not take more
        self._dtype, self._dev, self._B, self._Hkv, self._d = k.dtype, k.get_device(), B, Hkv, d


def _device_call(fn, name, dev, stream, *args):
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:  # the library launches on the current device
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status:
        _check(status, name)


def _paged_call(fn, name, cache, stream, *args):
    _device_call(fn, name, cache._dev, stream, *args)


def _paged_workspace(nbytes, cache, workspace, stream):
    """The caller's workspace, or a new one, its pointer and bytes."""
    if workspace is None:
        workspace = _scratch(nbytes() if callable(nbytes) else nbytes, cache.k.device, stream)
    elif workspace.get_device() != cache._dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def yoco_paged_attn_workspace_size(Hq, rows, cache: PagedKV) -> int:
    return lib.yoco_paged_attn_workspace_size(Hq, rows, cache.ref)


def _paged_cu(cu_rows, cache):
    if cu_rows.dtype != torch.int32 or cu_rows.shape != (cache._B + 1,) or cu_rows.get_device() != cache._dev or \
            not cu_rows.is_contiguous():
        raise ValueError("cu_rows must be a contiguous int32 [B + 1] on the cache's device")
    return cu_rows.data_ptr()


def _paged_source(t, name, cache, heads, rows):
    shape, stride = t.shape, t.stride()
    if t.dtype != cache._dtype or t.get_device() != cache._dev or len(shape) != 3 or shape[2] != cache._d or \
            stride[2] != 1 or (heads is not None and shape[1] != heads) or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be [rows, heads, {cache._d}] of {cache._dtype} with adjacent channels on the "
                         "cache's device")
    # (the stride of an axis of one element means nothing, and may be anything)
    return shape[0], shape[1], t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * shape[2], \
        stride[1] if shape[1] > 1 else shape[2]


def _paged_append_args(k, v, cache, cu_rows, q, q_out):
    rows, Hq, qo = None, 0, None
    kp = vp = qp = (None, 0, 0)
    if k is not None:
        rows, _, *kp = _paged_source(k, "k", cache, cache._Hkv, None)
    if v is not None:
        rows, _, *vp = _paged_source(v, "v", cache, cache._Hkv, rows)
    if q is not None:
        rows, Hq, *qp = _paged_source(q, "q", cache, None, rows)
        if q_out is None:
            q_out = q
        elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.get_device() != cache._dev or \
                not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous with q's shape and dtype on its device")
        qo = q_out.data_ptr()
    if rows is None:
        raise ValueError("neither k and v nor q given")
    cu = None if cu_rows is None else _paged_cu(cu_rows, cache)
    return *kp, *vp, *qp, qo, Hq, cu, rows, cache.ref


def yoco_paged_append(k, v, cache: PagedKV, cu_rows=None, q=None, q_out=None, workspace=None, stream=None):
    """k, v [rows, Hkv, d] (or both None), q [rows, Hq, d] or None, each with any strides
    that are multiples of 16 bytes; q_out [rows, Hq, d] (None: q in place).  cu_rows int32
    [B + 1], or None for one row per sequence."""
    args = _paged_append_args(k, v, cache, cu_rows, q, q_out)
    ws, wp, wn = _paged_workspace(256, cache, workspace, stream)
    _paged_call(lib.yoco_paged_append, "yoco_paged_append", cache, stream, *args, wp, wn)


def yoco_paged_append_rope(k, v, cache: PagedKV, rope: Rope, cu_rows=None, q=None, q_out=None, workspace=None,
                           stream=None):
    """yoco_paged_append with k and q turned as `rope` says (the cache's rope_base must be 0)."""
    args = _paged_append_args(k, v, cache, cu_rows, q, q_out)
    ws, wp, wn = _paged_workspace(256, cache, workspace, stream)
    _paged_call(lib.yoco_paged_append_rope, "yoco_paged_append_rope", cache, stream, *args, rope.ref, wp, wn)


def _paged_q(Q, O, cache):
    shape = Q.shape
    if len(shape) != 3 or shape[2] != cache._d or O.shape != shape or Q.dtype != cache._dtype or \
            O.dtype != cache._dtype or Q.get_device() != cache._dev or O.get_device() != cache._dev or \
            not Q.is_contiguous() or not O.is_contiguous():
        raise ValueError(f"Q and O must be contiguous [rows, Hq, {cache._d}] of {cache._dtype} on the cache's device")
    return shape[0], shape[1]


def _reach(slots):
    """A window or a number of sinks as the library's int: no sequence holds more than 2^30 slots, and
    ctypes would cut a larger number to its low 32 bits."""
    return max(-1, min(slots, 1 << 30))


def yoco_paged_attn_prefill(Q, cache: PagedKV, cu_rows, O, scale=None, window=0, sinks=0, workspace=None, stream=None):
    """Q, O [rows, Hq, d]; rows cu_rows[b] .. cu_rows[b + 1] - 1 are sequence b's newest."""
    rows, Hq = _paged_q(Q, O, cache)
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_attn_workspace_size(Hq, rows, cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_attn_prefill, "yoco_paged_attn_prefill", cache, stream, Q.data_ptr(), Hq,
                _paged_cu(cu_rows, cache), rows, cache.ref, cache._d ** -0.5 if scale is None else scale, _reach(window), _reach(sinks),
                O.data_ptr(), wp, wn)


def yoco_paged_attn_decode(Q, cache: PagedKV, O, scale=None, window=0, sinks=0, workspace=None, stream=None):
    """Q, O [B, Hq, d]: one row per sequence, at position seq_lens[b] - 1."""
    rows, Hq = _paged_q(Q, O, cache)
    if rows != cache._B:
        raise ValueError(f"Q has {rows} rows, the cache {cache._B} sequences")
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_attn_workspace_size(Hq, rows, cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_attn_decode, "yoco_paged_attn_decode", cache, stream, Q.data_ptr(), Hq, cache.ref,
                cache._d ** -0.5 if scale is None else scale, _reach(window), _reach(sinks), O.data_ptr(), wp, wn)


class PagedScores:
    """Scores other than scale q.k and masks other than causal ones, for the scored paged calls:
    a tanh cap, slopes fp32 [Hq] of a bias by distance, prefix int32 [B] (slots that every row of the
    sequence sees), doc_first int32 [rows] (the first slot of each row's document)."""

    def __init__(self, softcap=0.0, slopes=None, prefix=None, doc_first=None):
        for t, n, dt in ((slopes, "slopes", torch.float32), (prefix, "prefix", torch.int32),
                         (doc_first, "doc_first", torch.int32)):
            if t is not None:
                _need(t, n)
                if t.dtype != dt or t.dim() != 1:
                    raise ValueError(f"{n} must be a vector of {dt}")
        self.softcap, self.slopes, self.prefix, self.doc_first = softcap, slopes, prefix, doc_first
        self.c = _PagedScoresC(softcap, *(None if t is None else t.data_ptr() for t in (slopes, prefix, doc_first)))
        self.ref = ctypes.byref(self.c)

    def _check(self, cache, Hq, rows):
        for t, n, size in ((self.slopes, "slopes", Hq), (self.prefix, "prefix", cache._B),
                           (self.doc_first, "doc_first", rows)):
            if t is not None and (t.shape[0] != size or t.get_device() != cache._dev):
                raise ValueError(f"{n} must have {size} values on the cache's device")
        return self.ref


def yoco_paged_attn_prefill_scored(Q, cache: PagedKV, cu_rows, O, scores: PagedScores, scale=None, window=0, sinks=0,
                                   workspace=None, stream=None):
    """yoco_paged_attn_prefill with the scores and masks of `scores`."""
    rows, Hq = _paged_q(Q, O, cache)
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_attn_workspace_size(Hq, rows, cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_attn_prefill_scored, "yoco_paged_attn_prefill_scored", cache, stream, Q.data_ptr(), Hq,
                _paged_cu(cu_rows, cache), rows, cache.ref, scores._check(cache, Hq, rows),
                cache._d ** -0.5 if scale is None else scale, _reach(window), _reach(sinks), O.data_ptr(), wp, wn)


def yoco_paged_attn_decode_scored(Q, cache: PagedKV, O, scores: PagedScores, scale=None, window=0, sinks=0,
                                  workspace=None, stream=None):
    """yoco_paged_attn_decode with the scores and masks of `scores` (doc_first int32 [B])."""
    rows, Hq = _paged_q(Q, O, cache)
    if rows != cache._B:
        raise ValueError(f"Q has {rows} rows, the cache {cache._B} sequences")
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_attn_workspace_size(Hq, rows, cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_attn_decode_scored, "yoco_paged_attn_decode_scored", cache, stream, Q.data_ptr(), Hq,
                cache.ref, scores._check(cache, Hq, rows), cache._d ** -0.5 if scale is None else scale, _reach(window),
                _reach(sinks), O.data_ptr(), wp, wn)


# --------------------------------------------- the pages of a paged cache

def yoco_paged_pool_workspace_size(cache: PagedKV) -> int:
    return lib.yoco_paged_pool_workspace_size(cache.ref)


def _pool_ints(t, name, cache, size):
    if t.dtype != torch.int32 or t.get_device() != cache._dev or not t.is_contiguous() or t.dim() != 1 or \
            (size is not None and t.shape[0] != size):
        raise ValueError(f"{name} must be a contiguous int32 vector{'' if size is None else f' of {size}'} on the cache's device")
    return t.data_ptr()


def _pool_moves(moves, cache, most):
    if moves is None:
        return None
    if moves.dtype != torch.int32 or moves.get_device() != cache._dev or not moves.is_contiguous() or \
            moves.dim() != 2 or moves.shape[1] != 4 or moves.shape[0] < most + 1:
        raise ValueError(f"moves must be a contiguous int32 [>= {most + 1}, 4] on the cache's device")
    return moves.data_ptr()


def yoco_paged_resize(cache: PagedKV, refs, new_lens, moves=None, workspace=None, stream=None):
    """The sequences' lengths become new_lens (int32 [B], below 0: unchanged): cache.page_table,
    cache.seq_lens and refs (int32 [num_pages]) are written, shared pages that are written next are
    copied.  moves: int32 [>= B + 1, 4] for the list of copies, or None.
    A pool without room for all that grow raises nothing here (the call does not wait for the GPU):
    no sequence grows, seq_lens stay, and the workspace's status word says so.  Pass a workspace and
    ask yoco_workspace_status; one that the call makes itself takes its status word with it."""
    r, n = _pool_ints(refs, "refs", cache, cache.k.shape[0]), _pool_ints(new_lens, "new_lens", cache, cache._B)
    m = _pool_moves(moves, cache, cache._B)
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_pool_workspace_size(cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_resize, "yoco_paged_resize", cache, stream, cache.ref, r, n, m, wp, wn)


def yoco_paged_fork(cache: PagedKV, refs, src, dst, workspace=None, stream=None):
    """Empty sequences dst (int32 [n]) become what sequences src are, on the same pages.  Pairs that
    are left out are seen in the workspace's status word, as with yoco_paged_resize."""
    r, s = _pool_ints(refs, "refs", cache, cache.k.shape[0]), _pool_ints(src, "src", cache, None)
    d = _pool_ints(dst, "dst", cache, src.shape[0])
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_pool_workspace_size(cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_fork, "yoco_paged_fork", cache, stream, cache.ref, r, s, d, src.shape[0], wp, wn)


def yoco_paged_compact(cache: PagedKV, refs, moves=None, workspace=None, stream=None):
    """The pages in use become the pool's first ones.  moves: int32 [>= num_pages // 2 + 1, 4], or None."""
    r = _pool_ints(refs, "refs", cache, cache.k.shape[0])
    m = _pool_moves(moves, cache, cache.k.shape[0] // 2)
    ws, wp, wn = _paged_workspace(lambda: yoco_paged_pool_workspace_size(cache), cache, workspace, stream)
    _paged_call(lib.yoco_paged_compact, "yoco_paged_compact", cache, stream, cache.ref, r, m, wp, wn)


def yoco_paged_copy(cache: PagedKV, moves, stream=None):
    """Makes the copies of a list (int32 [n, 4]) that a resize or a compact of another cache with the
    same table wrote."""
    m = _pool_moves(moves, cache, 0)
    _paged_call(lib.yoco_paged_copy, "yoco_paged_copy", cache, stream, cache.ref, m, moves.shape[0] - 1)
