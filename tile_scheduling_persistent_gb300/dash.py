"""ctypes binding of libdash.so (C ABI in include/dash.h).

Argument marshalling only: every step of the backward pass runs in the
library's CUDA kernels.  Tensors are torch CUDA tensors (device memory and
streams come from PyTorch); the library fails loudly if it is missing.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import os
import struct
import threading

import numpy as np
import torch

from .inputs import SCHEDULE_IDS

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdash.so")

OK, ERR_ARG, ERR_CUDA, ERR_LAUNCH, ERR_TIMEOUT, ERR_DEADLOCK, ERR_NOMEM, ERR_DEVICE = 0, -1, -2, -3, -4, -5, -6, -7
ERR_SCRATCH, ERR_PAGE = -8, -9
_NAMES = {0: "DASH_OK", -1: "DASH_ERR_ARG", -2: "DASH_ERR_CUDA", -3: "DASH_ERR_LAUNCH", -4: "DASH_ERR_TIMEOUT",
          -5: "DASH_ERR_DEADLOCK", -6: "DASH_ERR_NOMEM", -7: "DASH_ERR_DEVICE", -8: "DASH_ERR_SCRATCH",
          -9: "DASH_ERR_PAGE"}

EXPORTS = (
    "dash_attn_bwd_preprocess", "dash_attn_bwd", "dash_dq_finalize", "dash_get_status", "dash_set_timeout_ns",
    "dash_release_workspaces", "dash_num_ctas", "dash_sim_schedule", "dash_sim_check_ranks",
    "dash_attn_bwd_debug", "dash_debug_tile_probe", "dash_attn_bwd_noalloc", "dash_select_schedule",
    "dash_attn_fwd", "dash_sim_schedule_band", "dash_attn_bwd_window", "dash_attn_fwd_window",
    "dash_sim_schedule_cross", "dash_attn_bwd_cross", "dash_attn_fwd_cross", "dash_head_split", "dash_key_blocks",
    "dash_noalloc_init", "dash_get_status_noalloc",
    "dash_rope", "dash_rope_freqs", "dash_kv_write", "dash_kv_read", "dash_attn_paged", "dash_attn_paged_workspace",
    "dash_get_status_paged",
)


class DashError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s failed: %s (%d)" % (what, _NAMES.get(code, "?"), code))
        self.code = code


class _DebugOpts(ctypes.Structure):
    _fields_ = [("order_log", ctypes.c_void_p), ("dq_partials", ctypes.c_void_p), ("cta_perm", ctypes.c_void_p),
                ("start_delay_ns", ctypes.c_void_p), ("ranks_host", ctypes.c_void_p),
                ("skip_table_check", ctypes.c_int), ("kernel_event_begin", ctypes.c_void_p),
                ("kernel_event_end", ctypes.c_void_p), ("wait_cycles", ctypes.c_void_p),
                ("event_trace", ctypes.c_void_p), ("window", ctypes.c_int), ("skv", ctypes.c_int),
                ("head_split", ctypes.c_int)]


# The structs of the rotary and paged calls (dash_heads, dash_kv_cache, dash_write_rope): packed natively, which
# costs a fifth of a ctypes.Structure on calls that last a few microseconds.
_HEADS = struct.Struct("@Piiqqq")
_CACHE = struct.Struct("@PPPPiiiii0P")
_WRITE_ROPE = struct.Struct("@PPiifPqqPqqi0P")


_lib = None


def lib():
    """Load libdash.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libdash.so is not built (run: python -m tile_scheduling_persistent_gb300.build)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, Z, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    L.dash_attn_bwd_preprocess.argtypes = [P, P, P, I, I, I, I, P]
    L.dash_attn_bwd.argtypes = [P] * 9 + [I] * 7 + [P]
    L.dash_attn_bwd_debug.argtypes = [P] * 9 + [I] * 7 + [P, ctypes.POINTER(_DebugOpts)]
    L.dash_attn_bwd_noalloc.argtypes = [P] * 9 + [I] * 7 + [P]
    L.dash_dq_finalize.argtypes = [P, P, Z, P]
    L.dash_get_status.argtypes = [P, ctypes.POINTER(I), ctypes.POINTER(I)]
    L.dash_get_status_noalloc.argtypes = [P, ctypes.POINTER(I), ctypes.POINTER(I)]
    L.dash_noalloc_init.argtypes = []
    L.dash_set_timeout_ns.argtypes = [ctypes.c_uint64]
    L.dash_release_workspaces.argtypes = []
    L.dash_num_ctas.argtypes = [I, ctypes.POINTER(I)]
    L.dash_sim_schedule.argtypes = [I] * 7 + [D, D, ctypes.POINTER(D), P, ctypes.POINTER(ctypes.c_int64)]
    L.dash_sim_schedule_band.argtypes = [I] * 7 + [D, D, ctypes.POINTER(D), P, ctypes.POINTER(ctypes.c_int64)]
    L.dash_sim_schedule_cross.argtypes = [I] * 7 + [D, D, ctypes.POINTER(D), P, ctypes.POINTER(ctypes.c_int64)]
    L.dash_sim_check_ranks.argtypes = [I] * 7 + [P]
    L.dash_debug_tile_probe.argtypes = [P] * 6 + [I, I] + [P] * 7
    L64 = ctypes.c_int64
    L.dash_rope.argtypes = [P, P, P, P, P, L64, P, I, I, ctypes.c_float, I, I, I, I, P]
    L.dash_rope_freqs.argtypes = [I, D, I, D, I, D, D, P, ctypes.POINTER(ctypes.c_float)]
    L.dash_kv_write.argtypes = [P, P, L64, L64, P, L64, L64, P, I, P, P]
    L.dash_kv_read.argtypes = [P, P, L64, I, P, P, P, L64, L64, L64, I, I, P]
    L.dash_attn_paged.argtypes = [P, L64, L64, P, P, L64, I, P, P, P, P, I, I, I, I, I, I, P, Z, P]
    L.dash_attn_paged_workspace.argtypes = [I, I, I, I, I, I, L64, ctypes.POINTER(Z)]
    L.dash_get_status_paged.argtypes = [P, ctypes.POINTER(I), ctypes.POINTER(I)]
    for name in EXPORTS:
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(rc, what):
    if rc != OK:
        raise DashError(rc, what)


def _sched(schedule):
    return SCHEDULE_IDS[schedule] if isinstance(schedule, str) else int(schedule)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t, dtype=None):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "expected a contiguous CUDA tensor"
    if dtype is not None:
        assert t.dtype == dtype, "expected %s, got %s" % (dtype, t.dtype)
    return ctypes.c_void_p(t.data_ptr())


def attn_bwd_preprocess(o, do, delta, stream=None):
    B, H, S, D = o.shape
    _check(lib().dash_attn_bwd_preprocess(_ptr(o, torch.bfloat16), _ptr(do, torch.bfloat16),
                                          _ptr(delta, torch.float32), B, H, S, D, _stream(stream)),
           "dash_attn_bwd_preprocess")


def _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule):
    B, Hq, S, D = q.shape
    Hkv = k.shape[1]
    bf, f32 = torch.bfloat16, torch.float32
    return [_ptr(q, bf), _ptr(k, bf), _ptr(v, bf), _ptr(o, bf), _ptr(do, bf), _ptr(lse, f32), _ptr(dq, f32),
            _ptr(dk, bf), _ptr(dv, bf), B, Hq, Hkv, S, D, int(bool(causal)), _sched(schedule)]


def attn_bwd(q, k, v, o, do, lse, dq, dk, dv, causal, schedule, stream=None, window=None):
    """dq (fp32 accumulator, zeroed by the library), dk, dv (bf16) <- backward.
    window: causal sliding window in tokens (needs causal=True), or None.
    k/v (and dk/dv) may be longer or shorter than q (full mask only)."""
    if k.shape[2] != q.shape[2]:
        assert not causal and window is None, "different lengths need a full mask"
        args = _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule)
        args[-3:-2] = [k.shape[2], q.shape[3]]   # (..., Sq, D, causal, sched) -> (..., Sq, Skv, D, sched)
        del args[-2]
        _check(lib().dash_attn_bwd_cross(*args, _stream(stream)), "dash_attn_bwd_cross")
        return
    if window is not None:
        assert causal, "a sliding window needs a causal mask"
        args = _bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule)
        args[-2] = int(window)   # the causal flag's slot carries the window
        _check(lib().dash_attn_bwd_window(*args, _stream(stream)), "dash_attn_bwd_window")
        return
    _check(lib().dash_attn_bwd(*_bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule), _stream(stream)),
           "dash_attn_bwd")


def attn_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, causal, schedule, stream=None):
    """attn_bwd for callers that cannot allocate: library scratch comes from a
    fixed device array (see dash_attn_bwd_noalloc in include/dash.h)."""
    _check(lib().dash_attn_bwd_noalloc(*_bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule),
                                       _stream(stream)), "dash_attn_bwd_noalloc")


def noalloc_init():
    """Set-up of attn_bwd_noalloc on the current device (scratch address, kernels loaded)."""
    _check(lib().dash_noalloc_init(), "dash_noalloc_init")


def get_status_noalloc(stream=None):
    """(code, info) of the last attn_bwd_noalloc on the current device; synchronizes `stream`."""
    code = ctypes.c_int(0)
    info = (ctypes.c_int * 4)()
    _check(lib().dash_get_status_noalloc(_stream(stream), ctypes.byref(code), info), "dash_get_status_noalloc")
    return code.value, list(info)


def attn_bwd_debug(q, k, v, o, do, lse, dq, dk, dv, causal, schedule, stream=None, order_log=None,
                   dq_partials=None, cta_perm=None, start_delay_ns=None, ranks_host=None, skip_table_check=False,
                   kernel_events=None, wait_cycles=None, event_trace=None, window=None, head_split=None):
    """head_split: None (the library decides), True (one task per query head)
    or False (one task per key/value head group)."""
    opts = _DebugOpts()
    opts.window = int(window) if window is not None else 0
    opts.head_split = 0 if head_split is None else (1 if head_split else 2)
    opts.skv = int(k.shape[2]) if k.shape[2] != q.shape[2] else 0
    opts.wait_cycles = _ptr(wait_cycles, torch.int64)
    opts.event_trace = _ptr(event_trace, torch.int64)
    if kernel_events is not None:
        opts.kernel_event_begin = ctypes.c_void_p(kernel_events[0].cuda_event)
        opts.kernel_event_end = ctypes.c_void_p(kernel_events[1].cuda_event)
    opts.order_log = _ptr(order_log, torch.int32)
    opts.dq_partials = _ptr(dq_partials, torch.float32)
    opts.cta_perm = _ptr(cta_perm, torch.int32)
    opts.start_delay_ns = _ptr(start_delay_ns, torch.int64)
    keep = None
    if ranks_host is not None:
        keep = np.ascontiguousarray(ranks_host, dtype=np.uint16)
        opts.ranks_host = keep.ctypes.data_as(ctypes.c_void_p)
    opts.skip_table_check = int(bool(skip_table_check))
    rc = lib().dash_attn_bwd_debug(*_bwd_args(q, k, v, o, do, lse, dq, dk, dv, causal, schedule),
                                   _stream(stream), ctypes.byref(opts))
    if keep is not None:
        torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
    _check(rc, "dash_attn_bwd_debug")


def dq_finalize(dq_accum, dq, stream=None):
    assert dq_accum.numel() == dq.numel()
    _check(lib().dash_dq_finalize(_ptr(dq_accum, torch.float32), _ptr(dq, torch.bfloat16), dq.numel(),
                                  _stream(stream)), "dash_dq_finalize")


def get_status(stream=None):
    code = ctypes.c_int(0)
    info = (ctypes.c_int * 4)()
    _check(lib().dash_get_status(_stream(stream), ctypes.byref(code), info), "dash_get_status")
    return code.value, list(info)


def set_timeout_ns(ns):
    _check(lib().dash_set_timeout_ns(int(ns)), "dash_set_timeout_ns")


def release_workspaces():
    """Gives back the device memory that calls keep: the library's, and attn_paged's of every thread and stream."""
    with _kept_lock:
        _kept.clear()
    _check(lib().dash_release_workspaces(), "dash_release_workspaces")


def attn_fwd(q, k, v, o, lse, causal, stream=None, window=None):
    """o (bf16 [B,Hq,S,D]) and lse (fp32 [B,Hq,S], natural log) <- forward.
    window: causal sliding window in tokens (needs causal=True), or None."""
    B, Hq, S, D = q.shape
    Hkv = k.shape[1]
    bf = torch.bfloat16
    ptrs = (_ptr(q, bf), _ptr(k, bf), _ptr(v, bf), _ptr(o, bf), _ptr(lse, torch.float32))
    if k.shape[2] != S:
        assert not causal and window is None, "different lengths need a full mask"
        _check(lib().dash_attn_fwd_cross(*ptrs, B, Hq, Hkv, S, k.shape[2], D, _stream(stream)), "dash_attn_fwd_cross")
        return
    if window is not None:
        assert causal, "a sliding window needs a causal mask"
        _check(lib().dash_attn_fwd_window(*ptrs, B, Hq, Hkv, S, D, int(window), _stream(stream)),
               "dash_attn_fwd_window")
        return
    _check(lib().dash_attn_fwd(*ptrs, B, Hq, Hkv, S, D, int(bool(causal)), _stream(stream)), "dash_attn_fwd")


def select_schedule(B, Hq, Hkv, S, D, causal):
    """Name of the deterministic schedule that schedule="auto" runs for this shape."""
    rc = lib().dash_select_schedule(B, Hq, Hkv, S, D, int(bool(causal)))
    _check(rc if rc < 0 else 0, "dash_select_schedule")
    return {v: k for k, v in SCHEDULE_IDS.items()}[rc]


def head_split(schedule, causal, B, Hq, Hkv, S, D, P, window=None, Skv=None):
    """True if the backward of this shape runs one task per query head (see
    dash_head_split); its accumulation order is then that of Hkv = Hq."""
    rc = lib().dash_head_split(_sched(schedule), int(bool(causal)), B, Hq, Hkv, S, D, int(window or 0),
                               int(Skv or 0), int(P))
    _check(rc if rc < 0 else 0, "dash_head_split")
    return rc == 1


def key_blocks(B, Hq, Hkv, Sq, Skv):
    """The number of key blocks the backward with key length Skv != Sq cuts
    the keys into (see dash_key_blocks); 1 = no split."""
    rc = lib().dash_key_blocks(int(B), int(Hq), int(Hkv), int(Sq), int(Skv))
    _check(rc if rc < 0 else 0, "dash_key_blocks")
    return rc


def task_heads(schedule, causal, B, Hq, Hkv, S, D, P, window=None, Skv=None):
    """The Hkv to simulate a backward run with: Hq when its tasks are split per
    query head, else Hkv."""
    return Hq if head_split(schedule, causal, B, Hq, Hkv, S, D, P, window, Skv) else Hkv


def num_ctas(device=None):
    dev = torch.cuda.current_device() if device is None else int(device)
    P = ctypes.c_int(0)
    _check(lib().dash_num_ctas(dev, ctypes.byref(P)), "dash_num_ctas")
    return P.value


def sim_schedule(schedule, causal, B, Hq, Hkv, n, P, c=1.0, r=1.0, turn_order=True, band=None, nkv=None):
    """Host DAG simulator: (makespan, turn order [B*Hq*n, nkv] or None, tasks).
    band: tile diagonals of a causal sliding window (None: no window);
    nkv: key/value tiles per head when they differ from n (full masks only)."""
    mk = ctypes.c_double(0.0)
    nt = ctypes.c_int64(0)
    nk = n if nkv is None else int(nkv)
    out = np.empty((B * Hq * n, nk), dtype=np.int32) if turn_order else None
    optr = out.ctypes.data_as(ctypes.c_void_p) if out is not None else None
    if nkv is not None:
        assert not causal and band is None, "S_q != S_kv needs a full mask"
        rc = lib().dash_sim_schedule_cross(_sched(schedule), B, Hq, Hkv, n, nk, P, float(c), float(r),
                                           ctypes.byref(mk), optr, ctypes.byref(nt))
    elif band is None:
        rc = lib().dash_sim_schedule(_sched(schedule), int(bool(causal)), B, Hq, Hkv, n, P, float(c), float(r),
                                     ctypes.byref(mk), optr, ctypes.byref(nt))
    else:
        assert causal, "a band needs a causal mask"
        rc = lib().dash_sim_schedule_band(_sched(schedule), B, Hq, Hkv, n, int(band), P, float(c), float(r),
                                          ctypes.byref(mk), optr, ctypes.byref(nt))
    _check(rc, "dash_sim_schedule")
    return mk.value, out, nt.value


def sim_check_ranks(schedule, causal, B, Hq, Hkv, n, P, ranks):
    arr = np.ascontiguousarray(ranks, dtype=np.uint16)
    return lib().dash_sim_check_ranks(_sched(schedule), int(bool(causal)), B, Hq, Hkv, n, P,
                                      arr.ctypes.data_as(ctypes.c_void_p))


def tile_probe(k, v, q, do, lse, delta, diag=False):
    """One pair through the kernel's building blocks; returns fp32 intermediates."""
    D = k.shape[-1]
    dev = k.device
    f = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)  # noqa: E731
    out = {name: f(128, 128) for name in ("sT", "pT", "dpT", "dsT")}
    out.update({name: f(128, D) for name in ("dv", "dk", "dq")})
    bf = torch.bfloat16
    _check(lib().dash_debug_tile_probe(_ptr(k, bf), _ptr(v, bf), _ptr(q, bf), _ptr(do, bf),
                                       _ptr(lse, torch.float32), _ptr(delta, torch.float32), D, int(bool(diag)),
                                       *[_ptr(out[n]) for n in ("sT", "pT", "dpT", "dsT", "dv", "dk", "dq")]),
           "dash_debug_tile_probe")
    return out


# ------------------------------------------------------------------ rotary positions, paged cache, paged attention
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "wave": 3, "ramp": 4}
_BF16, _F32, _I32, _I64, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _refuse(what, why):
    """Arguments that the C entry cannot see: tensor shapes, types, devices."""
    err = DashError(ERR_ARG, what)
    err.args = (err.args[0] + ": " + why,)
    raise err


def _device_stream(stream, what):
    """The current device, on which every tensor has to be, and the address of the stream (None: its current one)."""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, (_raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream)
    if stream.device_index != dev:
        _refuse(what, "the stream belongs to the current device")
    return dev, stream.cuda_stream


# These calls last a few microseconds, so the checks are written out where they are made: every method call on a tensor
# costs some 50 ns.  A stride of a dimension of size one is read as 0.
def _flat(t, dtype, dev, shape, what, name):
    """The address of a contiguous tensor."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(what, "%s is a contiguous %s tensor of shape %s on the current CUDA device" % (name, dtype, tuple(shape)))
    return t.data_ptr()


def _tokens(t, dev, shape, what, name):
    """The address and the token and head strides of a bf16 tensor [T, H, D]."""
    if t.dtype is not _BF16 or t.get_device() != dev or t.shape != shape or len(shape) != 3:
        _refuse(what, "%s is a bf16 tensor of shape %s on the current CUDA device" % (name, tuple(shape)))
    st, sh, sd = t.stride()
    if sd != 1:
        _refuse(what, "%s is contiguous in its last dimension" % name)
    return t.data_ptr(), (st if shape[0] > 1 else 0), (sh if shape[1] > 1 else 0)


def _heads(t, dev, what, name):
    """dash_heads of a [B, H, S, D] tensor, and its strides."""
    dtype = t.dtype
    shape = t.shape
    if len(shape) != 4 or t.get_device() != dev or (dtype is not _BF16 and dtype is not _F32):
        _refuse(what, "%s is a bf16 or fp32 tensor [B, H, S, D] on the current CUDA device" % name)
    sb, sh, ss, sd = t.stride()
    if sd != 1:
        _refuse(what, "%s is contiguous in its last dimension" % name)
    B, H, S, _ = shape
    if B == 1:
        sb = 0
    if H == 1:
        sh = 0
    if S == 1:
        ss = 0
    return _HEADS.pack(t.data_ptr(), dtype is _F32, H, sb, sh, ss), (sb, sh, ss)


def _cache(k, v, k_scale, v_scale, dev, what):
    """dash_kv_cache, its Hkv, page_size and D."""
    shape = k.shape
    if len(shape) != 4:
        _refuse(what, "the cache is [num_pages, Hkv, page_size, D]")
    N, H, page, D = shape
    dtype = k.dtype
    kp, vp = _flat(k, dtype, dev, shape, what, "k_cache"), _flat(v, dtype, dev, shape, what, "v_cache")
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            _refuse(what, "a bf16 cache has no scales")
        return _CACHE.pack(kp, vp, 0, 0, 0, N, page, H, D), H, page, D
    if dtype is not _E4M3 or k_scale is None or v_scale is None:
        _refuse(what, "the cache is bf16, or float8_e4m3fn with k_scale and v_scale")
    shape = (N, H, page)
    return _CACHE.pack(kp, vp, _flat(k_scale, _F32, dev, shape, what, "k_scale"),
                       _flat(v_scale, _F32, dev, shape, what, "v_scale"), 1, N, page, H, D), H, page, D


def _table(block_table, B, dev, what):
    """The address of an int32 tensor [B, pages], its row stride and width."""
    shape = block_table.shape
    if block_table.dtype is not _I32 or block_table.get_device() != dev or len(shape) != 2 or shape[0] != B:
        _refuse(what, "block_table is an int32 tensor [B, pages] on the current CUDA device")
    row, col = block_table.stride()
    if col != 1 and shape[1] > 1:
        _refuse(what, "block_table is contiguous in its last dimension")
    return block_table.data_ptr(), (row if B > 1 else 0), shape[1]


def _freqs(inv_freq, what):
    """inv_freq as something to keep alive, its address and the rotated width."""
    if not isinstance(inv_freq, torch.Tensor):
        inv_freq = torch.as_tensor(np.ascontiguousarray(inv_freq, dtype=np.float64))
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() >= 0 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        _refuse(what, "inv_freq is a contiguous float64 vector on the host")
    return inv_freq, inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def rope_freqs(rot, base=10000.0, scaling="none", scale=1.0, trained=0, lo=1.0, hi=4.0):
    """(inv_freq, factor): the float64 radians per position of the rot/2 pairs of
    a rotary embedding, and the factor that goes with its long-context scaling
    ("none", "linear", "base", "wave", "ramp"; see dash_rope_freqs)."""
    out = torch.empty(max(int(rot) // 2, 1), dtype=torch.float64)
    factor = ctypes.c_float(1.0)
    _check(lib().dash_rope_freqs(int(rot), float(base), ROPE_SCALINGS[scaling], float(scale), int(trained), float(lo),
                                 float(hi), out.data_ptr(), ctypes.byref(factor)), "dash_rope_freqs")
    return out, factor.value


def rope(x, y, inv_freq, positions=None, x2=None, y2=None, interleaved=False, factor=1.0, inverse=False, stream=None):
    """y <- rotary positions of x [B, H, S, D] (bf16 or fp32, any strides but the
    last), and y2 of x2 with the same positions: int32 [S], [B, S] or None (0, 1, ...).
    inv_freq: float64 [rot/2] on the host (rope_freqs); inverse=True is the
    backward (y = dL/dx for x = dL/dy).  y may be x."""
    what = "dash_rope"
    dev, st = _device_stream(stream, what)
    keep, freqs, rot = _freqs(inv_freq, what)
    a, b = _heads(x, dev, what, "x")[0], _heads(y, dev, what, "y")[0]
    shape = x.shape
    B, _, S, D = shape
    if shape != y.shape:
        _refuse(what, "y has the shape of x")
    a2 = b2 = None
    if x2 is not None and y2 is not None:
        a2, b2 = _heads(x2, dev, what, "x2")[0], _heads(y2, dev, what, "y2")[0]
        shape = x2.shape
        if shape != y2.shape or shape[0] != B or shape[2] != S or shape[3] != D:
            _refuse(what, "x2 and y2 are [B, H2, S, D]")
    elif x2 is not None or y2 is not None:
        _refuse(what, "x2 and y2 go together")
    pos, pos_b = None, 0
    if positions is not None:
        if positions.shape == (S,):
            pos = _flat(positions, _I32, dev, (S,), what, "positions")
        else:
            pos, pos_b, width = _table(positions, B, dev, what)
            if width != S:
                _refuse(what, "positions is [S] or [B, S]")
    _check(lib().dash_rope(a, b, a2, b2, pos, pos_b, freqs, rot, bool(interleaved), factor, bool(inverse), B, S, D, st),
           what)


def kv_write(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, inv_freq=None, positions=None,
             interleaved=False, factor=1.0, q=None, q_out=None, stream=None):
    """Write new tokens' k, v [T, Hkv, D] (bf16, any token and head strides) into
    the pages [num_pages, Hkv, page_size, D] at slots int64 [T] (page * page_size +
    offset, no two the same; negative: skipped); an e4m3 cache (torch.float8_e4m3fn) quantises each
    vector with its own scale.  inv_freq and positions int32 [T]: k is rotated on
    the way (see rope), and q [T, Hq, D] into q_out."""
    what = "dash_kv_write"
    dev, st = _device_stream(stream, what)
    c, Hkv, _, D = _cache(k_cache, v_cache, k_scale, v_scale, dev, what)
    T = k.shape[0]
    shape = (T, Hkv, D)
    kp, kt, kh = _tokens(k, dev, shape, what, "k")
    vp, vt, vh = _tokens(v, dev, shape, what, "v")
    sp = _flat(slots, _I64, dev, (T,), what, "slots")
    r = keep = None
    if inv_freq is not None:
        if positions is None:
            _refuse(what, "a rotation needs positions")
        keep, freqs, rot = _freqs(inv_freq, what)
        qp = qt = qh = op = ot = oh = Hq = 0
        if q is not None:
            if q_out is None or q.dim() != 3:
                _refuse(what, "q and q_out are [T, Hq, D]")
            Hq = q.shape[1]
            shape = (T, Hq, D)
            qp, qt, qh = _tokens(q, dev, shape, what, "q")
            op, ot, oh = _tokens(q_out, dev, shape, what, "q_out")
        elif q_out is not None:
            _refuse(what, "q_out needs q")
        r = _WRITE_ROPE.pack(freqs, _flat(positions, _I32, dev, (T,), what, "positions"), rot, bool(interleaved), factor,
                             qp, qt, qh, op, ot, oh, Hq)
    elif q is not None or q_out is not None or positions is not None:
        _refuse(what, "q, q_out and positions need inv_freq")
    _check(lib().dash_kv_write(c, kp, kt, kh, vp, vt, vh, sp, T, r, st), what)


def kv_read(k_cache, v_cache, block_table, lens, k, v, k_scale=None, v_scale=None, stream=None):
    """k, v [B, Hkv, S, D] (bf16, equal strides) <- the first lens[b] cached tokens of
    each sequence; rows past lens[b] are left as they were.  block_table int32
    [B, pages], lens int32 [B]."""
    what = "dash_kv_read"
    dev, st = _device_stream(stream, what)
    c, Hkv, _, D = _cache(k_cache, v_cache, k_scale, v_scale, dev, what)
    (_, ks), (_, vs) = _heads(k, dev, what, "k"), _heads(v, dev, what, "v")
    shape = k.shape
    B, H, S, d = shape
    if H != Hkv or d != D or v.shape != shape or ks != vs or k.dtype is not _BF16 or v.dtype is not _BF16:
        _refuse(what, "k and v are bf16 [B, Hkv, S, D] with equal strides")
    tp, ts, pages = _table(block_table, B, dev, what)
    _check(lib().dash_kv_read(c, tp, ts, pages, _flat(lens, _I32, dev, (B,), what, "lens"), k.data_ptr(), v.data_ptr(),
                              *ks, B, S, st), what)


_KEPT_BYTES, _KEPT_TOTAL = 32 << 20, 256 << 20   # of one workspace, and of all
_kept = collections.OrderedDict()                # (thread, device, stream): workspace, the last used at the end
_kept_lock = threading.RLock()                   # (a finalizer that runs in here may call attn_paged)


def _workspace(n, dev, st):
    """n bytes for a call on the current stream st.  Up to _KEPT_BYTES are kept, for each thread and stream: an allocation
    between launches costs 7 us, as much as all else in the call.  Calls of one thread on one stream run one after
    another; a captured call, whose replays do not keep to its stream, gets memory of its graph's own.  All that is kept is
    at most _KEPT_TOTAL: the longest unused go first (the allocator hands them to later work of their stream alone, so a
    call in flight may still use them; those of a thread that ended serve the next of its number, or go that way)."""
    if n > _KEPT_BYTES or torch.cuda.is_current_stream_capturing():
        return torch.empty(n, dtype=torch.uint8, device=dev)
    key = threading.get_ident(), dev, st
    try:   # (without the lock: another thread can only take the entry away)
        w = _kept[key]
        if w.numel() >= n:
            _kept.move_to_end(key)
            return w
    except KeyError:
        pass
    w = torch.empty(max(n, 1 << 20), dtype=torch.uint8, device=dev)
    with _kept_lock:
        _kept[key] = w
        _kept.move_to_end(key)
        total = sum(t.numel() for t in _kept.values())
        while total > _KEPT_TOTAL:
            total -= _kept.popitem(last=False)[1].numel()
    return w


@functools.lru_cache(maxsize=4096)   # a function of the sizes alone
def attn_paged_workspace(B, T, Hq, Hkv, D, max_q, max_kv):
    """Bytes of workspace attn_paged needs; max_kv = pages per sequence * page_size."""
    out = ctypes.c_size_t(0)
    _check(lib().dash_attn_paged_workspace(B, T, Hq, Hkv, D, max_q, max_kv, ctypes.byref(out)),
           "dash_attn_paged_workspace")
    return out.value


def attn_paged(q, k_cache, v_cache, block_table, kv_lens, o, cu_q=None, max_q=None, lse=None, causal=True, window=None,
               k_scale=None, v_scale=None, workspace=None, stream=None):
    """o [T, Hq, D] (and lse fp32 [T, Hq]) <- attention of each sequence's newest
    tokens q [T, Hq, D] over its kv_lens[b] cached tokens, the new ones among them
    (see dash_attn_paged).  cu_q int32 [B+1] are the sequences' first rows (None:
    T / B rows each) and max_q bounds their new tokens (None: T with cu_q, else
    T / B).  workspace: uint8 tensor of attn_paged_workspace bytes (None: the
    binding's own, kept for this thread and stream where it is small and the call
    is not being captured, 256 MiB in all; release_workspaces frees it)."""
    what = "dash_attn_paged"
    dev, st = _device_stream(stream, what)
    c, Hkv, page, D = _cache(k_cache, v_cache, k_scale, v_scale, dev, what)
    shape = q.shape
    if len(shape) != 3 or shape[2] != D:
        _refuse(what, "q is [T, Hq, D]")
    T, Hq, _ = shape
    qp, qt, qh = _tokens(q, dev, shape, what, "q")
    op = _flat(o, _BF16, dev, shape, what, "o")
    lp = _flat(lse, _F32, dev, (T, Hq), what, "lse") if lse is not None else None
    B = kv_lens.shape[0]
    tp, ts, pages = _table(block_table, B, dev, what)
    lens = _flat(kv_lens, _I32, dev, (B,), what, "kv_lens")
    cp = _flat(cu_q, _I32, dev, (B + 1,), what, "cu_q") if cu_q is not None else None
    if max_q is None:
        max_q = T if cu_q is not None or B == 0 else T // B
    if window is None:
        window = 0
    elif not causal or window < 1:
        _refuse(what, "a sliding window has at least one token, and a causal mask")
    if workspace is None:
        wn, wp = attn_paged_workspace(B, T, Hq, Hkv, D, max_q, pages * page), None
        if wn:
            if stream is None:
                workspace = _workspace(wn, dev, st)
            else:
                with torch.cuda.stream(stream):   # the allocator's reuse then follows this stream
                    workspace = torch.empty(wn, dtype=torch.uint8, device=q.device)
            wp = workspace.data_ptr()
    else:
        wn = workspace.numel()
        wp = _flat(workspace, torch.uint8, dev, (wn,), what, "workspace")
    _check(lib().dash_attn_paged(qp, qt, qh, c, tp, ts, pages, lens, cp, op, lp, B, T, Hq, max_q, bool(causal), window,
                                 wp, wn, st), what)


def get_status_paged(stream=None):
    """(code, info) of an error that kv_write, kv_read or attn_paged recorded on the
    current device, which is then cleared; synchronizes `stream`.  Errors of several
    operators come one a call, until the code is 0 (see dash_get_status_paged)."""
    code = ctypes.c_int(0)
    info = (ctypes.c_int * 4)()
    _check(lib().dash_get_status_paged(_stream(stream), ctypes.byref(code), info), "dash_get_status_paged")
    return code.value, list(info)
