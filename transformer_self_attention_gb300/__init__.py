"""GB300 (sm_103a) self-attention forward: Python binding of libattn.so.

Argument marshalling only.  Every step of the forward pass runs in the CUDA
kernels of libattn.so; there is no CPU or PyTorch fallback.  If the library is
missing (not built), importing this module raises.

Low-level functions mirror the C ABI of ``include/attn.h`` (same names, integer
pointers); :class:`Attention` wraps a handle for torch tensors.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_DEVICE_TIMEOUT, ATTN_ERR_OOM = range(6)
MASK_FULL, MASK_CAUSAL, MASK_SLIDING, MASK_CAUSAL_SLIDING, MASK_LOCAL_GLOBAL = range(5)
ATTN_BF16, ATTN_F32, ATTN_FP8_E4M3 = 0, 1, 2
TILE = 128
WORK_INTS = 8
LIST_FULL = 1 << 16  # ATTN_LIST_FULL: the FULL flag of a backward list entry
WORK_GLOBAL_COLS, WORK_GLOBAL_ROWS, WORK_HAS_GLOBAL_ROWS = 1, 2, 4

EXPORTED = ("attn_create", "attn_forward", "attn_destroy", "attn_status_string", "attn_schedule_host",
            "attn_poll_device_error", "attn_set_watchdog", "attn_forward_noalloc", "attn_selftest_exp2",
            "attn_decode_create", "attn_decode_forward", "attn_decode_poll_device_error", "attn_decode_destroy",
            "attn_decode_schedule_host", "attn_decode_set_grid_limit", "attn_set_alibi",
            "attn_decode_set_alibi", "attn_set_fp8_descale", "attn_kv_schedule_host",
            "attn_backward", "attn_bwd_dq_schedule_host", "attn_set_bias", "attn_decode_set_merge_mode",
            "attn_decode_launch_count", "attn_selftest_device_once", "attn_forward_noalloc_poll_error",
            "attn_forward_noalloc_set_watchdog", "attn_bwd_lg_lists_host",
            "attn_rope_create", "attn_rope_frequencies", "attn_rope_forward", "attn_rope_backward",
            "attn_rope_destroy", "attn_cache_create", "attn_cache_write", "attn_cache_read",
            "attn_cache_poll_device_error", "attn_cache_destroy", "attn_paged_create", "attn_paged_forward",
            "attn_paged_set_grid_limit", "attn_paged_set_watchdog", "attn_paged_destroy", "attn_paged_split_host")
NOALLOC_SCRATCH_BYTES = 8 << 20
DECODE_MAX_BATCH = 1024
DECODE_MAX_ROWS = 64
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
CACHE_ERR_POSITION, CACHE_ERR_PAGE, CACHE_ERR_WAIT = 1, 2, 4


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {attn_status_string(status)} (status {status})")
        self.status = status


class attn_rows(ctypes.Structure):
    """Rows of contiguous elements: data pointer and strides (in elements) over batch, head and position."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_s", ctypes.c_longlong)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libattn.so not built at {LIB_PATH}; run __graft_entry__.build() "
                          "(the library has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    I, P, F, LL = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong
    lib.attn_create.argtypes = [ctypes.POINTER(P), I, I, I, I, I, I, F, I, I, P, I]
    lib.attn_create.restype = I
    lib.attn_forward.argtypes = [P, P, P, P, P, P, P]
    lib.attn_forward.restype = I
    lib.attn_destroy.argtypes = [P]
    lib.attn_destroy.restype = I
    lib.attn_status_string.argtypes = [I]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_schedule_host.argtypes = [I, I, I, I, I, I, P, I, P, I, ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.attn_schedule_host.restype = I
    lib.attn_poll_device_error.argtypes = [P, ctypes.POINTER(I)]
    lib.attn_poll_device_error.restype = I
    lib.attn_set_watchdog.argtypes = [P, LL, I]
    lib.attn_set_watchdog.restype = I
    lib.attn_set_alibi.argtypes = [P, P]
    lib.attn_set_alibi.restype = I
    lib.attn_decode_set_alibi.argtypes = [P, P]
    lib.attn_decode_set_alibi.restype = I
    lib.attn_set_fp8_descale.argtypes = [P, F, F, F]
    lib.attn_set_fp8_descale.restype = I
    lib.attn_kv_schedule_host.argtypes = [I, I, I, P, I, ctypes.POINTER(I)]
    lib.attn_kv_schedule_host.restype = I
    lib.attn_backward.argtypes = [P] * 11
    lib.attn_backward.restype = I
    lib.attn_bwd_dq_schedule_host.argtypes = [I, I, I, I, I, I, I, P, I, ctypes.POINTER(I)]
    lib.attn_bwd_dq_schedule_host.restype = I
    lib.attn_bwd_lg_lists_host.argtypes = [I, I, P, I, P, I, P, ctypes.POINTER(I)]
    lib.attn_bwd_lg_lists_host.restype = I
    lib.attn_set_bias.argtypes = [P, P, I, I, ctypes.c_long]
    lib.attn_set_bias.restype = I
    lib.attn_decode_set_merge_mode.argtypes = [P, I]
    lib.attn_decode_set_merge_mode.restype = I
    lib.attn_decode_launch_count.argtypes = [P, ctypes.POINTER(I)]
    lib.attn_decode_launch_count.restype = I
    lib.attn_forward_noalloc.argtypes = [I, I, I, I, I, F, I, I, P, I, P, P, P, P, P, P]
    lib.attn_forward_noalloc.restype = I
    lib.attn_forward_noalloc_poll_error.argtypes = [ctypes.POINTER(I)]
    lib.attn_forward_noalloc_poll_error.restype = I
    lib.attn_forward_noalloc_set_watchdog.argtypes = [ctypes.c_longlong, I]
    lib.attn_forward_noalloc_set_watchdog.restype = I
    lib.attn_selftest_exp2.argtypes = [P, P, I, P]
    lib.attn_selftest_exp2.restype = I
    lib.attn_selftest_device_once.argtypes = []
    lib.attn_selftest_device_once.restype = I
    lib.attn_decode_create.argtypes = [ctypes.POINTER(P), I, I, I, I, I, I, F, I, I]
    lib.attn_decode_create.restype = I
    lib.attn_decode_forward.argtypes = [P, P, P, P, P, P, P, P]
    lib.attn_decode_forward.restype = I
    lib.attn_decode_poll_device_error.argtypes = [P, ctypes.POINTER(I)]
    lib.attn_decode_poll_device_error.restype = I
    lib.attn_decode_destroy.argtypes = [P]
    lib.attn_decode_destroy.restype = I
    lib.attn_decode_schedule_host.argtypes = [I, I, I, I, I, I, P, I, ctypes.POINTER(I), P, P]
    lib.attn_decode_schedule_host.restype = I
    lib.attn_decode_set_grid_limit.argtypes = [P, I]
    lib.attn_decode_set_grid_limit.restype = I
    D, R = ctypes.c_double, ctypes.POINTER(attn_rows)
    rope = [P, I, I, I, I, R, R, I, R, R, P, LL, LL, P]
    for name, args in (("attn_rope_create", [ctypes.POINTER(P), I, I, I, D, I, D, I, D, D, D]),
                       ("attn_rope_frequencies", [P, P, P]), ("attn_rope_forward", rope),
                       ("attn_rope_backward", rope), ("attn_rope_destroy", [P]),
                       ("attn_cache_create", [ctypes.POINTER(P), I, I, I, I, I, P, P]),
                       ("attn_cache_write", [P, I, I, R, R, P, LL, I, P, P, P, I, R, R, P]),
                       ("attn_cache_read", [P, I, I, I, R, R, P, LL, I, P, P]),
                       ("attn_cache_poll_device_error", [P, ctypes.POINTER(I)]), ("attn_cache_destroy", [P]),
                       ("attn_paged_create", [ctypes.POINTER(P), I, I, I, I, I, F, I, I]),
                       ("attn_paged_forward", [P, P, P, P, LL, I, P, P, P, P]),
                       ("attn_paged_set_grid_limit", [P, I]), ("attn_paged_set_watchdog", [P, LL, I]),
                       ("attn_paged_destroy", [P]),
                       ("attn_paged_split_host", [I, I, I, I, I, I, I, P, I, ctypes.POINTER(I), P, I,
                                                  ctypes.POINTER(I)])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I
    return lib


_lib = _load()


def _int_array(xs: Optional[Sequence[int]]):
    xs = list(xs or [])
    arr = (ctypes.c_int * max(len(xs), 1))(*xs)
    return arr, len(xs)


# ---------------------------------------------------------------- C ABI, same names

def attn_status_string(status: int) -> str:
    return _lib.attn_status_string(int(status)).decode()


def attn_create(B, Hq, Hkv, S, d_k, dtype, scale, kind, window=0, global_idx=None) -> int:
    """Returns a handle (int); raises AttnError on a non-OK status."""
    h = ctypes.c_void_p()
    g, ng = _int_array(global_idx)
    st = _lib.attn_create(ctypes.byref(h), int(B), int(Hq), int(Hkv), int(S), int(d_k), int(dtype),
                          float(scale), int(kind), int(window), ctypes.cast(g, ctypes.c_void_p) if ng else None, ng)
    if st != ATTN_OK:
        raise AttnError(st, "attn_create")
    return h.value


def attn_forward(handle: int, q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int = 0,
                 stream: int = 0) -> int:
    """Enqueue the forward pass; returns the status (does not raise)."""
    return _lib.attn_forward(handle, q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr or None, stream or None)


def attn_destroy(handle: int) -> int:
    return _lib.attn_destroy(handle)


def attn_poll_device_error(handle: int):
    code = ctypes.c_int(0)
    st = _lib.attn_poll_device_error(handle, ctypes.byref(code))
    return st, code.value


def _float_array(xs):
    xs = [float(x) for x in xs]
    return (ctypes.c_float * max(len(xs), 1))(*xs)


def attn_set_alibi(handle: int, slopes=None) -> int:
    """ALiBi bias -slopes[a] |i - j| on later forwards of this handle (None removes it); returns the status."""
    if slopes is None:
        return _lib.attn_set_alibi(handle, None)
    return _lib.attn_set_alibi(handle, ctypes.cast(_float_array(slopes), ctypes.c_void_p))


def attn_set_watchdog(handle: int, limit_ns: int, withhold: int = 0) -> int:
    return _lib.attn_set_watchdog(handle, int(limit_ns), int(withhold))


def attn_forward_noalloc(B, Hq, Hkv, S, d_k, scale, kind, window, global_idx, q_ptr, k_ptr, v_ptr, o_ptr,
                         lse_ptr=0, stream=0) -> int:
    """The bf16 forward pass without any device allocation (fixed library-owned scratch); returns the status.

    For callers that cannot allocate device memory.  Calls that overlap on the GPU race on the shared
    scratch; the first call on a device should come before any stream capture.
    """
    g, ng = _int_array(global_idx)
    return _lib.attn_forward_noalloc(int(B), int(Hq), int(Hkv), int(S), int(d_k), float(scale), int(kind),
                                     int(window), ctypes.cast(g, ctypes.c_void_p) if ng else None, ng,
                                     q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr or None, stream or None)


def attn_forward_noalloc_poll_error():
    """(status, code): synchronise, read and clear the error word of attn_forward_noalloc's scratch."""
    code = ctypes.c_int(0)
    st = _lib.attn_forward_noalloc_poll_error(ctypes.byref(code))
    return st, code.value


def attn_forward_noalloc_set_watchdog(limit_ns: int, withhold: int = 0) -> int:
    """Test hook: wait limit and V-withholding of attn_forward_noalloc's kernels (process-wide)."""
    return _lib.attn_forward_noalloc_set_watchdog(int(limit_ns), int(withhold))


def attn_selftest_exp2(x_ptr: int, y_ptr: int, n: int, stream: int = 0) -> int:
    """Test hook: the library's FMA-pipe exp2 applied elementwise (device float arrays)."""
    return _lib.attn_selftest_exp2(x_ptr, y_ptr, int(n), stream or None)


def attn_selftest_device_once() -> int:
    """Host-only test hook of the per-device kernel set-up registry (0 = every check held)."""
    return _lib.attn_selftest_device_once()


def attn_schedule_host(B, Hq, Hkv, S, kind, window=0, global_idx=None):
    """Host-only schedule: (items int32 [n, 8], n_first).  Raises AttnError on bad arguments."""
    g, ng = _int_array(global_idx)
    gp = ctypes.cast(g, ctypes.c_void_p) if ng else None
    n, n_first = ctypes.c_int(0), ctypes.c_int(0)
    st = _lib.attn_schedule_host(int(B), int(Hq), int(Hkv), int(S), int(kind), int(window), gp, ng, None, 0,
                                 ctypes.byref(n), ctypes.byref(n_first))
    if st != ATTN_OK:
        raise AttnError(st, "attn_schedule_host")
    items = np.zeros((max(n.value, 1), WORK_INTS), dtype=np.int32)
    st = _lib.attn_schedule_host(int(B), int(Hq), int(Hkv), int(S), int(kind), int(window), gp, ng,
                                 items.ctypes.data_as(ctypes.c_void_p), n.value, ctypes.byref(n),
                                 ctypes.byref(n_first))
    if st != ATTN_OK:
        raise AttnError(st, "attn_schedule_host")
    return items[: n.value], n_first.value


def attn_kv_schedule_host(S, kind, window=0):
    """Backward key-tile schedule (host only): int32 [n, 8].  Raises AttnError."""
    n = ctypes.c_int(0)
    st = _lib.attn_kv_schedule_host(int(S), int(kind), int(window), None, 0, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv_schedule_host")
    items = np.zeros((max(n.value, 1), WORK_INTS), dtype=np.int32)
    st = _lib.attn_kv_schedule_host(int(S), int(kind), int(window), items.ctypes.data_as(ctypes.c_void_p), n.value,
                                    ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_kv_schedule_host")
    return items[: n.value]


def attn_bwd_lg_lists_host(S, window, globals_idx):
    """The backward's per-tile partner lists under local + global (host only): (list, offsets),
    int32 arrays; entries t | LIST_FULL.  Raises AttnError."""
    g = np.ascontiguousarray(np.asarray(list(globals_idx), dtype=np.int32).reshape(-1))
    gp = g.ctypes.data_as(ctypes.c_void_p) if g.size else None
    n = ctypes.c_int(0)
    st = _lib.attn_bwd_lg_lists_host(int(S), int(window), gp, int(g.size), None, 0, None, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_lg_lists_host")
    lst = np.zeros(max(n.value, 1), dtype=np.int32)
    off = np.zeros((S + TILE - 1) // TILE + 1, dtype=np.int32)
    st = _lib.attn_bwd_lg_lists_host(int(S), int(window), gp, int(g.size), lst.ctypes.data_as(ctypes.c_void_p),
                                     n.value, off.ctypes.data_as(ctypes.c_void_p), ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_lg_lists_host")
    return lst[: n.value], off


def attn_bwd_dq_schedule_host(B, Hq, Hkv, S, d_k, kind, window=0):
    """Work items of the backward's dQ launch (host only): int32 [n, 8].  Raises AttnError."""
    n = ctypes.c_int(0)
    args = (int(B), int(Hq), int(Hkv), int(S), int(d_k), int(kind), int(window))
    st = _lib.attn_bwd_dq_schedule_host(*args, None, 0, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_dq_schedule_host")
    items = np.zeros((max(n.value, 1), WORK_INTS), dtype=np.int32)
    st = _lib.attn_bwd_dq_schedule_host(*args, items.ctypes.data_as(ctypes.c_void_p), n.value, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_dq_schedule_host")
    return items[: n.value]


# ---------------------------------------------------------------- decode (key/value cache)

def attn_decode_create(B, Hq, Hkv, S_q, S_cap, d_k, scale, kind, window=0) -> int:
    """Returns a decode handle (int); raises AttnError on a non-OK status."""
    h = ctypes.c_void_p()
    st = _lib.attn_decode_create(ctypes.byref(h), int(B), int(Hq), int(Hkv), int(S_q), int(S_cap), int(d_k),
                                 float(scale), int(kind), int(window))
    if st != ATTN_OK:
        raise AttnError(st, "attn_decode_create")
    return h.value


def attn_decode_forward(handle: int, q_ptr: int, k_ptr: int, v_ptr: int, cache_len, o_ptr: int,
                        lse_ptr: int = 0, stream: int = 0) -> int:
    """Enqueue one decode step (cache_len: host sequence of B ints); returns the status."""
    lens, n = _int_array(cache_len)
    return _lib.attn_decode_forward(handle, q_ptr, k_ptr, v_ptr, ctypes.cast(lens, ctypes.c_void_p), o_ptr,
                                    lse_ptr or None, stream or None)


def attn_decode_poll_device_error(handle: int):
    code = ctypes.c_int(0)
    st = _lib.attn_decode_poll_device_error(handle, ctypes.byref(code))
    return st, code.value


def attn_decode_destroy(handle: int) -> int:
    return _lib.attn_decode_destroy(handle)


def attn_decode_schedule_host(B, Hkv, S_q, S_cap, kind, window, cache_len, n_sm):
    """Host-only decode work split: (n_cta, tile_prefix int32 [B + 1], share int64 [n_cta + 1]).
    CTA k takes the tile-list indices [share[k], share[k + 1]).  Raises AttnError."""
    lens, n = _int_array(cache_len)
    n_cta = ctypes.c_int(0)
    prefix = np.zeros(int(B) + 1, dtype=np.int32)
    share = np.zeros(max(1, int(n_sm)) + 1, dtype=np.int64)
    st = _lib.attn_decode_schedule_host(int(B), int(Hkv), int(S_q), int(S_cap), int(kind), int(window),
                                        ctypes.cast(lens, ctypes.c_void_p), int(n_sm), ctypes.byref(n_cta),
                                        prefix.ctypes.data_as(ctypes.c_void_p),
                                        share.ctypes.data_as(ctypes.c_void_p))
    if st != ATTN_OK:
        raise AttnError(st, "attn_decode_schedule_host")
    return n_cta.value, prefix, share[:n_cta.value + 1].copy()


class DecodeAttention:
    """A decode plan: S_q new query rows per sequence against a key/value cache.

    Q: [B, Hq, S_q, d] bf16; K, V (the cache): [B, Hkv, S_cap, d] bf16; cache_len: B host ints.
    Row i of sequence b sits at position cache_len[b] - S_q + i.  Returns (O like Q, LSE float32
    [B, Hq, S_q]).
    """

    def __init__(self, B, Hq, Hkv, S_q, S_cap, d, scale=None, kind=MASK_CAUSAL, window=0):
        import math
        self.shape = (int(B), int(Hq), int(Hkv), int(S_q), int(S_cap), int(d))
        self.scale = float(scale) if scale is not None else 1.0 / math.sqrt(d)
        self.kind, self.window = int(kind), int(window)
        self.handle = attn_decode_create(B, Hq, Hkv, S_q, S_cap, d, self.scale, self.kind, self.window)

    def close(self):
        if getattr(self, "handle", None):
            attn_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __call__(self, Q, K, V, cache_len, O=None, LSE=None, stream=None, want_lse=True):
        import torch
        B, Hq, Hkv, S_q, S_cap, d = self.shape
        for name, t, shape in (("Q", Q, (B, Hq, S_q, d)), ("K", K, (B, Hkv, S_cap, d)), ("V", V, (B, Hkv, S_cap, d))):
            if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or tuple(t.shape) != shape:
                raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor of shape {shape}")
        if O is None:
            O = torch.empty_like(Q)
        if LSE is None and want_lse:
            LSE = torch.empty((B, Hq, S_q), dtype=torch.float32, device=Q.device)
        if stream is None:
            stream = torch.cuda.current_stream(Q.device)
        st = attn_decode_forward(self.handle, Q.data_ptr(), K.data_ptr(), V.data_ptr(), list(cache_len),
                                 O.data_ptr(), LSE.data_ptr() if LSE is not None else 0, stream.cuda_stream)
        if st != ATTN_OK:
            raise AttnError(st, "attn_decode_forward")
        return O, LSE

    def poll_device_error(self):
        return attn_decode_poll_device_error(self.handle)

    def set_alibi(self, slopes=None):
        """Add the ALiBi score bias -slopes[a] |t - j| (one slope per query head); None removes it."""
        if slopes is None:
            st = _lib.attn_decode_set_alibi(self.handle, None)
        else:
            if len(slopes) != self.shape[1]:
                raise ValueError("one slope per query head")
            st = _lib.attn_decode_set_alibi(self.handle, ctypes.cast(_float_array(slopes), ctypes.c_void_p))
        if st != ATTN_OK:
            raise AttnError(st, "attn_decode_set_alibi")

    def set_grid_limit(self, max_ctas: int):
        """Test hook: at most max_ctas CTAs per launch (long shares on small problems)."""
        st = _lib.attn_decode_set_grid_limit(self.handle, int(max_ctas))
        if st != ATTN_OK:
            raise AttnError(st, "attn_decode_set_grid_limit")

    def launch_count(self) -> int:
        """Kernels the last call enqueued (1, or 2 with the merge kernel)."""
        n = ctypes.c_int(0)
        st = _lib.attn_decode_launch_count(self.handle, ctypes.byref(n))
        if st != ATTN_OK:
            raise AttnError(st, "attn_decode_launch_count")
        return n.value

    def set_merge_mode(self, mode: int):
        """Where split units are merged: 0 auto, 1 in the decode kernel, 2 by the merge kernel."""
        st = _lib.attn_decode_set_merge_mode(self.handle, int(mode))
        if st != ATTN_OK:
            raise AttnError(st, "attn_decode_set_merge_mode")


# ---------------------------------------------------------------- rotary positions, paged cache, paged decode

def _int(x) -> int:
    """An argument of C type int, which ctypes would cut to 32 bits without a word."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{x} does not fit a C int")
    return x


def attn_rope_create(d, rot, layout=0, base=10000.0, scaling=0, factor=1.0, original_len=0, beta_fast=32.0,
                     beta_slow=1.0, amplitude=0.0) -> int:
    """Returns a rope handle (int; host only); raises AttnError on a non-OK status."""
    h = ctypes.c_void_p()
    st = _lib.attn_rope_create(ctypes.byref(h), _int(d), _int(rot), _int(layout), float(base), _int(scaling),
                               float(factor), _int(original_len), float(beta_fast), float(beta_slow),
                               float(amplitude))
    if st != ATTN_OK:
        raise AttnError(st, "attn_rope_create")
    return h.value


def attn_rope_frequencies(handle: int, rot: int):
    """(frequencies float64 [rot / 2], amplitude) of a rope handle."""
    f, amp = np.zeros(int(rot) // 2), ctypes.c_double(0)
    st = _lib.attn_rope_frequencies(handle, f.ctypes.data_as(ctypes.c_void_p),
                                    ctypes.cast(ctypes.byref(amp), ctypes.c_void_p))
    if st != ATTN_OK:
        raise AttnError(st, "attn_rope_frequencies")
    return f, amp.value


def attn_rope_forward(handle, dtype, B, S, Hq, Q, Q_out, Hk=0, K=None, K_out=None, positions=0, pos_stride_b=0,
                      pos_stride_s=0, stream=0) -> int:
    """Rotate rows (attn_rows structures); returns the status."""
    return _lib.attn_rope_forward(handle, dtype, B, S, Hq, Q, Q_out, Hk, K, K_out, positions or None, pos_stride_b,
                                  pos_stride_s, stream or None)


def attn_rope_backward(handle, dtype, B, S, Hq, dQ_out, dQ, Hk=0, dK_out=None, dK=None, positions=0, pos_stride_b=0,
                       pos_stride_s=0, stream=0) -> int:
    """Gradients of attn_rope_forward; returns the status."""
    return _lib.attn_rope_backward(handle, dtype, B, S, Hq, dQ_out, dQ, Hk, dK_out, dK, positions or None,
                                   pos_stride_b, pos_stride_s, stream or None)


def attn_rope_destroy(handle: int) -> int:
    return _lib.attn_rope_destroy(handle)


def attn_cache_create(n_pages, Hkv, page, d, dtype, pages_ptr, scales_ptr=0) -> int:
    """Returns a cache handle (int) over the given device buffers; raises AttnError."""
    h = ctypes.c_void_p()
    st = _lib.attn_cache_create(ctypes.byref(h), _int(n_pages), _int(Hkv), _int(page), _int(d), _int(dtype),
                                pages_ptr or None, scales_ptr or None)
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache_create")
    return h.value


def attn_cache_write(handle, B, S_new, K, V, table_ptr, table_stride, max_pages, len_ptr, new_len_ptr=0, rope=0, Hq=0,
                     Q=None, Q_out=None, stream=0) -> int:
    """Append rows to the cache (attn_rows structures, device pointers); returns the status."""
    return _lib.attn_cache_write(handle, B, S_new, K, V, table_ptr, table_stride, max_pages, len_ptr,
                                 new_len_ptr or None, rope or None, Hq, Q, Q_out, stream or None)


def attn_cache_read(handle, B, S, first, K, V, table_ptr, table_stride, max_pages, len_ptr, stream=0) -> int:
    """Positions of every sequence as dense rows; returns the status."""
    return _lib.attn_cache_read(handle, B, S, first, K, V, table_ptr, table_stride, max_pages, len_ptr,
                                stream or None)


def attn_cache_poll_device_error(handle: int):
    code = ctypes.c_int(0)
    st = _lib.attn_cache_poll_device_error(handle, ctypes.byref(code))
    return st, code.value


def attn_cache_destroy(handle: int) -> int:
    return _lib.attn_cache_destroy(handle)


def attn_paged_create(B, Hq, Hkv, S_q, d, scale, kind, window=0) -> int:
    """Returns a paged decode handle (int); raises AttnError on a non-OK status."""
    h = ctypes.c_void_p()
    st = _lib.attn_paged_create(ctypes.byref(h), _int(B), _int(Hq), _int(Hkv), _int(S_q), _int(d), float(scale),
                                _int(kind), _int(window))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_create")
    return h.value


def attn_paged_forward(handle, cache, q_ptr, table_ptr, table_stride, max_pages, len_ptr, o_ptr, lse_ptr=0,
                       stream=0) -> int:
    """Enqueue one decode step over a paged cache; returns the status."""
    return _lib.attn_paged_forward(handle, cache, q_ptr, table_ptr, table_stride, max_pages, len_ptr, o_ptr,
                                   lse_ptr or None, stream or None)


def attn_paged_set_grid_limit(handle: int, max_ctas: int) -> int:
    return _lib.attn_paged_set_grid_limit(handle, _int(max_ctas))


def attn_paged_set_watchdog(handle: int, limit_ns: int, withhold: int = 0) -> int:
    return _lib.attn_paged_set_watchdog(handle, int(limit_ns), _int(withhold))


def attn_paged_destroy(handle: int) -> int:
    return _lib.attn_paged_destroy(handle)


def attn_paged_split_host(B, Hkv, S_q, d, dtype, kind, window, cache_len, grid):
    """Host-only split of the paged decode: (n_cta, int32 [parts, 8]: CTA, sequence, kv head, first key block,
    one past the last, key blocks of the unit, first and last CTA of the unit).  Raises AttnError."""
    lens, n_lens = _int_array(cache_len)
    if n_lens != B:
        raise ValueError(f"cache_len must have {B} entries")
    n_cta, n = ctypes.c_int(0), ctypes.c_int(0)
    args = (_int(B), _int(Hkv), _int(S_q), _int(d), _int(dtype), _int(kind), _int(window),
            ctypes.cast(lens, ctypes.c_void_p), _int(grid))
    st = _lib.attn_paged_split_host(*args, ctypes.byref(n_cta), None, 0, ctypes.byref(n))
    parts = np.zeros((max(n.value, 1), 8), dtype=np.int32)
    if st == ATTN_OK:
        st = _lib.attn_paged_split_host(*args, ctypes.byref(n_cta), parts.ctypes.data_as(ctypes.c_void_p), n.value,
                                        ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_split_host")
    return n_cta.value, parts[:n.value]


torch = None  # the torch module, once a class below is used (the C ABI functions above do without it)


def _need_torch():
    global torch
    if torch is None:
        import torch as module
        torch = module
    return torch


def _rows(name, t, shape, dtype, device, out=False):
    """attn_rows of a tensor view [B, H, S, d] (shape: a tuple) whose last dimension is contiguous, on CUDA device
    number `device`; out: it is written, so its rows must not be one another."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{device}")
    sb, sh, ss, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    B, H, S, _ = shape
    # the stride of a dimension of one may be anything
    if B == 1:
        sb = 0
    if H == 1:
        sh = 0
    if S == 1:
        ss = 0
    if out and ((B > 1 and not sb) or (H > 1 and not sh) or (S > 1 and not ss)):
        raise ValueError(f"{name} is written and must not be an expanded tensor")
    return attn_rows(t.data_ptr(), sb, sh, ss)


def _new(shape, dtype, device, stream, zero=False):
    """A tensor for the results of a call on `stream` (None: the current one).  It comes from that stream's own memory,
    which work still pending on the current stream does not touch, and is reported to the allocator as used by the
    current stream too, where the caller goes on with it."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _new_rows(t, H, S, d):
    """attn_rows of a tensor [B, H, S, d] allocated here."""
    return attn_rows(t.data_ptr(), H * S * d, S * d, d)


def _int32(name, t, shape, device):
    """Pointer of a contiguous int32 tensor."""
    if t.dtype is not torch.int32 or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on cuda:{device}")
    return t.data_ptr()


def _call(device, stream, fn, args, used):
    """fn(*args, stream) with CUDA device number `device` current; `used`: the tensors of the call, reported to the
    caching allocator when the stream is not the current one.  Returns fn's status."""
    old = torch._C._cuda_getDevice()
    if old != device:
        torch.cuda.set_device(device)
    try:
        raw = torch._C._cuda_getCurrentRawStream(device)
        if stream is not None and stream.cuda_stream != raw:
            raw = stream.cuda_stream
            for t in used:
                if t is not None:
                    t.record_stream(stream)
        return fn(*args, raw)
    finally:
        if old != device:
            torch.cuda.set_device(old)


class RotaryPositions:
    """Rotary position embedding of Q and K (``attn_rope_*``), and its gradient.

    d: head width (a multiple of 16, at most 256); rotary_dim: how many of its elements are rotated, the first
    ones (default d); layout: pairs "half" (p, p + rotary_dim / 2) or "interleaved" (2p, 2p + 1); scaling: "none",
    "linear", "ntk" or "yarn" for contexts ``factor`` times longer ("yarn" with original_len, beta_fast,
    beta_slow); amplitude: factor on the rotated elements (default 1, or YaRN's 0.1 ln factor + 1).
    """

    def __init__(self, d, rotary_dim=None, layout="half", base=10000.0, scaling="none", factor=1.0, original_len=0,
                 beta_fast=32.0, beta_slow=1.0, amplitude=None):
        if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
            raise ValueError(f"layout is one of {sorted(ROPE_LAYOUTS)}, scaling one of {sorted(ROPE_SCALINGS)}")
        if amplitude is not None and not amplitude > 0:
            raise ValueError("amplitude must be positive")
        _need_torch()
        self.d, self.rotary_dim = int(d), int(d if rotary_dim is None else rotary_dim)
        self.handle = attn_rope_create(d, self.rotary_dim, ROPE_LAYOUTS[layout], base, ROPE_SCALINGS[scaling], factor,
                                       original_len, beta_fast, beta_slow, amplitude or 0.0)

    def close(self):
        if getattr(self, "handle", None):
            attn_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def frequencies(self):
        """(radians per position of each pair, float64 array; amplitude)."""
        return attn_rope_frequencies(self.handle, self.rotary_dim)

    def __call__(self, Q, K=None, positions=None, Q_out=None, K_out=None, stream=None):
        """Rotated Q [B, Hq, S, d] and K [B, Hk, S, d] (bf16 or float32 views, last dimension contiguous, rows
        16-byte aligned) by positions, int32 [B, S] or [S] (default 0 .. S - 1).  Returns (Q_out, K_out), or
        Q_out without K; the outputs may be the inputs."""
        return self._apply(_lib.attn_rope_forward, "attn_rope_forward", Q, K, positions, Q_out, K_out, stream)

    def backward(self, dQ_out, dK_out=None, positions=None, dQ=None, dK=None, stream=None):
        """Gradients with respect to the unrotated Q and K from those with respect to the rotated ones."""
        return self._apply(_lib.attn_rope_backward, "attn_rope_backward", dQ_out, dK_out, positions, dQ, dK, stream)

    def _apply(self, fn, name, Q, K, positions, Q_out, K_out, stream):
        dtype, device, shape = Q.dtype, Q.get_device(), Q.shape
        if (dtype is not torch.bfloat16 and dtype is not torch.float32) or len(shape) != 4 or shape[3] != self.d \
                or shape[1] < 1 or device < 0:
            raise ValueError(f"Q must be a CUDA bfloat16 or float32 tensor [B, Hq, S, {self.d}], Hq > 0")
        B, Hq, S, d = shape
        q = _rows("Q", Q, shape, dtype, device)
        if Q_out is None:
            Q_out = _new(shape, dtype, Q.device, stream)
            qo = _new_rows(Q_out, Hq, S, d)
        else:
            qo = _rows("Q_out", Q_out, shape, dtype, device, True)
        Hk, k, ko = 0, None, None
        if K is not None:
            if K.dim() != 4 or K.shape[1] < 1:
                raise ValueError(f"K must be a tensor [B, Hk, S, {d}] with at least one head")
            Hk = K.shape[1]
            shape = (B, Hk, S, d)
            k = _rows("K", K, shape, dtype, device)
            if K_out is None:
                K_out = _new(shape, dtype, Q.device, stream)
                ko = _new_rows(K_out, Hk, S, d)
            else:
                ko = _rows("K_out", K_out, shape, dtype, device, True)
        pos, pb, ps = None, 0, 0
        if positions is not None:
            if positions.dtype is not torch.int32 or positions.get_device() != device \
                    or (positions.shape != (B, S) and positions.shape != (S,)):
                raise ValueError(f"positions must be an int32 tensor of shape {(B, S)} or {(S,)} on {Q.device}")
            pos = positions.data_ptr()
            pb, ps = positions.stride() if positions.dim() == 2 else (0, positions.stride(0))
        if B * S:
            st = _call(device, stream, fn, (self.handle, ATTN_BF16 if dtype is torch.bfloat16 else ATTN_F32, B, S, Hq, q,
                                            qo, Hk, k, ko, pos, pb, ps), (Q, K, positions, Q_out, K_out))
            if st != ATTN_OK:
                raise AttnError(st, name)
        return Q_out if K is None else (Q_out, K_out)


class PagedCache:
    """A key/value cache in pages (``attn_cache_*``).

    pages: [n_pages, Hkv, 2, page, d] bfloat16 or float8_e4m3fn, keys and values at index 0 and 1; scales (E4M3):
    uint8 [n_pages, Hkv, page / 16, 2, 16], the biased exponent of each row's factor.  Both are allocated (zeroed)
    unless given, and stay the caller's to use.  page_table: int32 CUDA [B, max_pages]; cache_len: int32 CUDA [B], the
    positions of each sequence with the rows of the call counted in.  Both are read on the device.
    """

    def __init__(self, n_pages, Hkv, page, d, dtype="bf16", pages=None, scales=None, device=None):
        _need_torch()
        kinds = {"bf16": (ATTN_BF16, torch.bfloat16), "e4m3": (ATTN_FP8_E4M3, torch.float8_e4m3fn)}
        if dtype not in kinds:
            raise ValueError(f"dtype is one of {sorted(kinds)}")
        code, tdt = kinds[dtype]
        self.shape, self.dtype = (int(n_pages), int(Hkv), int(page), int(d)), dtype
        n_pages, Hkv, page, d = self.shape
        if min(self.shape) < 1 or page % 16:
            raise ValueError("n_pages, Hkv and d must be positive, page a positive multiple of 16")
        want = (n_pages, Hkv, 2, page, d)
        made = pages is None or (dtype == "e4m3" and scales is None)
        if pages is None:
            pages = torch.zeros(want, dtype=torch.uint8 if dtype == "e4m3" else tdt,
                                device=device or torch.device("cuda", torch.cuda.current_device()))
            pages = pages.view(tdt)
        if tuple(pages.shape) != want or pages.dtype != tdt or not pages.is_cuda or not pages.is_contiguous():
            raise ValueError(f"pages must be a contiguous CUDA {tdt} tensor of shape {want}")
        self.device, self._device = pages.device, pages.get_device()
        if dtype == "e4m3":
            want = (n_pages, Hkv, page // 16, 2, 16)
            if scales is None:
                scales = torch.zeros(want, dtype=torch.uint8, device=self.device)
            if (tuple(scales.shape) != want or scales.dtype != torch.uint8 or scales.device != self.device
                    or not scales.is_contiguous()):
                raise ValueError(f"scales must be a contiguous uint8 tensor of shape {want} on {self.device}")
        elif scales is not None:
            raise ValueError("a bf16 cache has no scales")
        self.pages, self.scales = pages, scales
        if made:  # the zeros are there before the first call, on whatever stream that is
            torch.cuda.current_stream(self.device).synchronize()
        with torch.cuda.device(self.device):
            self.handle = attn_cache_create(n_pages, Hkv, page, d, code, pages.data_ptr(),
                                            0 if scales is None else scales.data_ptr())

    def close(self):
        if getattr(self, "handle", None):
            with torch.cuda.device(self.device):
                attn_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _table(self, page_table, cache_len):
        """(B, arguments of the C calls: table pointer, row stride, pages a row, lengths pointer)."""
        if (page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.get_device() != self._device
                or page_table.shape[1] < 1 or page_table.stride(1) != 1):
            raise ValueError(f"page_table must be an int32 tensor [B, max_pages] with contiguous rows on {self.device}")
        B, wide = page_table.shape
        return B, (page_table.data_ptr(), page_table.stride(0), wide,
                   _int32("cache_len", cache_len, (B,), self._device))

    def write(self, K, V, page_table, cache_len, new_len=None, rope=None, Q=None, Q_out=None, stream=None):
        """Append K, V [B, Hkv, S_new, d] (bf16 views): row i < new_len[b] (int32 CUDA [B]; default S_new) of
        sequence b goes to position cache_len[b] - new_len[b] + i.  With ``rope`` (RotaryPositions) the keys, and
        Q [B, Hq, S_new, d] if given, are rotated by those positions; returns the rotated Q, or None."""
        _, Hkv, _, d = self.shape
        device = self._device
        B, table = self._table(page_table, cache_len)
        if K.dim() != 4:
            raise ValueError(f"K must be a tensor [{B}, {Hkv}, S_new, {d}]")
        S = K.shape[2]
        shape = (B, Hkv, S, d)
        k = _rows("K", K, shape, torch.bfloat16, device)
        v = _rows("V", V, shape, torch.bfloat16, device)
        if rope is not None and (rope.d != d or not rope.handle):
            raise ValueError("rope is for another head width, or closed")
        Hq, q, qo = 0, None, None
        if Q is not None:
            if rope is None:
                raise ValueError("Q is only taken to be rotated: give rope")
            if Q.dim() != 4 or Q.shape[1] < 1:
                raise ValueError(f"Q must be a tensor [{B}, Hq, {S}, {d}] with at least one head")
            Hq = Q.shape[1]
            shape = (B, Hq, S, d)
            q = _rows("Q", Q, shape, torch.bfloat16, device)
            if Q_out is None:
                Q_out = _new(shape, torch.bfloat16, self.device, stream)
                qo = _new_rows(Q_out, Hq, S, d)
            else:
                qo = _rows("Q_out", Q_out, shape, torch.bfloat16, device, True)
        new = None if new_len is None else _int32("new_len", new_len, (B,), device)
        if B:
            st = _call(device, stream, _lib.attn_cache_write,
                       (self.handle, B, S, k, v, *table, new, None if rope is None else rope.handle, Hq, q, qo),
                       (K, V, Q, Q_out, page_table, cache_len, new_len, self.pages, self.scales))
            if st != ATTN_OK:
                raise AttnError(st, "attn_cache_write")
        return Q_out if Q is not None else None

    def read(self, page_table, cache_len, first=0, length=None, K=None, V=None, stream=None):
        """Positions first .. first + length - 1 of every sequence as dense (K, V), bf16 [B, Hkv, length, d].
        Rows at or past cache_len[b] are left as they were (zeros in tensors allocated here)."""
        _, Hkv, _, d = self.shape
        B, table = self._table(page_table, cache_len)
        if length is None:
            if K is None and V is None:
                raise ValueError("give length, or the tensors to fill")
            length = (K if K is not None else V).shape[2]
        shape = (B, Hkv, int(length), d)
        # (a new tensor's zeros come before the rows: they are written on the same stream)
        if K is None:
            K = _new(shape, torch.bfloat16, self.device, stream, zero=True)
        if V is None:
            V = _new(shape, torch.bfloat16, self.device, stream, zero=True)
        k = _rows("K", K, shape, torch.bfloat16, self._device, True)
        v = _rows("V", V, shape, torch.bfloat16, self._device, True)
        if B:
            st = _call(self._device, stream, _lib.attn_cache_read,
                       (self.handle, B, int(length), _int(first), k, v, *table), (K, V, page_table, cache_len, self.pages, self.scales))
            if st != ATTN_OK:
                raise AttnError(st, "attn_cache_read")
        return K, V

    def poll_device_error(self):
        """(status, code): synchronise; code has the CACHE_ERR_* bits recorded since the last poll."""
        with torch.cuda.device(self.device):
            return attn_cache_poll_device_error(self.handle)


class PagedDecodeAttention:
    """A decode plan over a PagedCache: S_q new query rows per sequence, lengths and page table on the device.

    Q: [B, Hq, S_q, d] bf16; row i of sequence b sits at position cache_len[b] - S_q + i, its own key and value
    already written.  Returns (O like Q, LSE float32 [B, Hq, S_q]); a row that sees no key gives zeros and -inf.
    """

    def __init__(self, B, Hq, Hkv, S_q, d, scale=None, kind=MASK_CAUSAL, window=0, device=None):
        import math
        _need_torch()
        self.shape = (int(B), int(Hq), int(Hkv), int(S_q), int(d))
        self.scale = float(scale) if scale is not None else 1.0 / math.sqrt(d)
        self.kind, self.window = int(kind), int(window)
        with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
            self._device = torch.cuda.current_device()
            self.device = torch.device("cuda", self._device)
            self.handle = attn_paged_create(B, Hq, Hkv, S_q, d, self.scale, self.kind, self.window)

    def close(self):
        if getattr(self, "handle", None):
            with torch.cuda.device(self.device):
                attn_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __call__(self, Q, cache, page_table, cache_len, O=None, LSE=None, stream=None, want_lse=True):
        B, Hq, _, S_q, d = self.shape
        rows, table = cache._table(page_table, cache_len)
        if rows != B:
            raise ValueError(f"page_table must have {B} rows")
        shape = (B, Hq, S_q, d)
        for name, t, want, dt in (("Q", Q, shape, torch.bfloat16), ("O", O, shape, torch.bfloat16),
                                  ("LSE", LSE, shape[:3], torch.float32)):
            if (t is not None or name == "Q") and (t.dtype is not dt or t.get_device() != self._device
                                                   or t.shape != want or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {want} on {self.device}")
        if O is None:
            O = _new(shape, torch.bfloat16, self.device, stream)
        if LSE is None and want_lse:
            LSE = _new(shape[:3], torch.float32, self.device, stream)
        st = _call(self._device, stream, _lib.attn_paged_forward,
                   (self.handle, cache.handle, Q.data_ptr(), *table, O.data_ptr(), None if LSE is None else LSE.data_ptr()),
                   (Q, O, LSE, page_table, cache_len, cache.pages, cache.scales))
        if st != ATTN_OK:
            raise AttnError(st, "attn_paged_forward")
        return O, LSE

    def set_grid_limit(self, max_ctas: int):
        """Test hook: at most max_ctas CTAs per launch (long shares on small problems)."""
        st = attn_paged_set_grid_limit(self.handle, max_ctas)
        if st != ATTN_OK:
            raise AttnError(st, "attn_paged_set_grid_limit")

    def set_watchdog(self, limit_ns: int, withhold: int = 0):
        """Test hook: the limit of every bounded wait; with withhold = n > 0 a loading warp with n key blocks to load
        behind one another stops in front of the n-th."""
        st = attn_paged_set_watchdog(self.handle, limit_ns, withhold)
        if st != ATTN_OK:
            raise AttnError(st, "attn_paged_set_watchdog")


# ---------------------------------------------------------------- torch convenience

class Attention:
    """A plan (handle) for one problem shape; call with CUDA torch tensors.

    Q: [B, Hq, S, d], K/V: [B, Hkv, S, d], contiguous, bf16 (or fp32 for dtype="f32").
    Returns (O, LSE) with O like Q and LSE float32 [B, Hq, S].
    """

    def __init__(self, B, Hq, Hkv, S, d, dtype="bf16", scale=None, kind=MASK_CAUSAL, window=0,
                 global_idx=None):
        import math
        self.shape = (int(B), int(Hq), int(Hkv), int(S), int(d))
        self.dtype = dtype
        self.scale = float(scale) if scale is not None else 1.0 / math.sqrt(d)
        self.kind, self.window = int(kind), int(window)
        self.global_idx = list(global_idx or [])
        code = {"bf16": ATTN_BF16, "f32": ATTN_F32, "e4m3": ATTN_FP8_E4M3}[dtype]
        self.handle = attn_create(B, Hq, Hkv, S, d, code, self.scale, self.kind, self.window, self.global_idx)

    def close(self):
        if getattr(self, "handle", None):
            attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __call__(self, Q, K, V, O=None, LSE=None, stream=None, want_lse=True):
        import torch
        B, Hq, Hkv, S, d = self.shape
        tdt = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[self.dtype]
        for name, t, h in (("Q", Q, Hq), ("K", K, Hkv), ("V", V, Hkv)):
            if not t.is_cuda or t.dtype != tdt or not t.is_contiguous() or tuple(t.shape) != (B, h, S, d):
                raise ValueError(f"{name} must be a contiguous CUDA {tdt} tensor of shape {(B, h, S, d)}")
        if O is None:
            O = torch.empty(Q.shape, dtype=torch.bfloat16 if self.dtype == "e4m3" else Q.dtype, device=Q.device)
        if LSE is None and want_lse:
            LSE = torch.empty((B, Hq, S), dtype=torch.float32, device=Q.device)
        if stream is None:
            stream = torch.cuda.current_stream(Q.device)
        st = attn_forward(self.handle, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                          LSE.data_ptr() if LSE is not None else 0, stream.cuda_stream)
        if st != ATTN_OK:
            raise AttnError(st, "attn_forward")
        return O, LSE

    def poll_device_error(self):
        return attn_poll_device_error(self.handle)

    def set_watchdog(self, limit_ns: int, withhold: int = 0):
        st = attn_set_watchdog(self.handle, limit_ns, withhold)
        if st != ATTN_OK:
            raise AttnError(st, "attn_set_watchdog")

    def backward(self, Q, K, V, O, LSE, dO, dQ=None, dK=None, dV=None, stream=None):
        """Gradients (dQ, dK, dV) of this plan's forward for the output gradient dO (bf16 tensors;
        O and LSE from the forward call)."""
        import torch
        if dQ is None:
            dQ = torch.empty_like(Q)
        if dK is None:
            dK = torch.empty_like(K)
        if dV is None:
            dV = torch.empty_like(V)
        for name, t in (("O", O), ("dO", dO), ("dQ", dQ)):
            if t.shape != Q.shape or t.dtype != Q.dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous tensor like Q")
        if stream is None:
            stream = torch.cuda.current_stream(Q.device)
        st = _lib.attn_backward(self.handle, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(),
                                dO.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), stream.cuda_stream)
        if st != ATTN_OK:
            raise AttnError(st, "attn_backward")
        return dQ, dK, dV

    def set_fp8_descale(self, descale_q: float, descale_k: float, descale_v: float):
        """Per-tensor factors of E4M3 inputs (real value = factor x stored value)."""
        st = _lib.attn_set_fp8_descale(self.handle, float(descale_q), float(descale_k), float(descale_v))
        if st != ATTN_OK:
            raise AttnError(st, "attn_set_fp8_descale")

    def set_alibi(self, slopes=None):
        """Add the ALiBi score bias -slopes[a] |i - j| (one slope per query head); None removes it."""
        if slopes is not None and len(slopes) != self.shape[1]:
            raise ValueError("one slope per query head")
        st = attn_set_alibi(self.handle, slopes)
        if st != ATTN_OK:
            raise AttnError(st, "attn_set_alibi")

    def set_bias(self, bias=None):
        """Add a bias matrix b_ij to the scores: a CUDA bf16 tensor [Bb, Hb, S, ld] (Bb in {1, B},
        Hb in {1, Hq}, ld >= S a multiple of 8; a 3-D [Hb, S, ld] or 2-D [S, ld] tensor is taken as
        Bb = 1 / Hb = 1).  The tensor is kept referenced by the plan; None removes the bias."""
        if bias is None:
            st = _lib.attn_set_bias(self.handle, None, 0, 0, 0)
            self._bias = None
        else:
            import torch
            t = bias
            while t.dim() < 4:
                t = t.unsqueeze(0)
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("bias must be a contiguous CUDA bf16 tensor")
            Bb, Hb, S, ld = t.shape
            if S != self.shape[3]:
                raise ValueError("bias rows must be the sequence length")
            st = _lib.attn_set_bias(self.handle, t.data_ptr(), int(Bb), int(Hb), int(ld))
            self._bias = t if st == ATTN_OK else None
        if st != ATTN_OK:
            raise AttnError(st, "attn_set_bias")
