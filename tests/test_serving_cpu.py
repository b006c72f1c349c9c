"""Rotary positions, paged cache and paged attention without a GPU: frequencies
against their formulas, every refusal that needs no device, the oracle itself."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class Heads(ctypes.Structure):       # dash_heads
    _fields_ = [("data", P), ("fp32", I), ("heads", I), ("stride_b", Z), ("stride_h", Z), ("stride_s", Z)]


class Cache(ctypes.Structure):       # dash_kv_cache
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("type", I), ("num_pages", I), ("page_size", I),
                ("Hkv", I), ("D", I)]


class WriteRope(ctypes.Structure):   # dash_write_rope
    _fields_ = [("inv_freq", P), ("positions", P), ("rot", I), ("interleaved", I), ("factor", ctypes.c_float), ("q", P),
                ("q_stride_t", Z), ("q_stride_h", Z), ("q_out", P), ("q_out_stride_t", Z), ("q_out_stride_h", Z), ("Hq", I)]


def test_the_bindings_layouts_are_the_structs():
    for packed, cls in ((dash._HEADS, Heads), (dash._CACHE, Cache), (dash._WRITE_ROPE, WriteRope)):
        assert packed.size == ctypes.sizeof(cls)
        values = list(range(1, len(cls._fields_) + 1))
        got = cls.from_buffer_copy(packed.pack(*values))
        assert [getattr(got, f) for f, _ in cls._fields_] == values


OK, BAD = 4096, 4098   # an aligned and a misaligned address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dash.lib()


SCALED = [("none", dict()), ("linear", dict(scale=4.0)), ("base", dict(scale=8.0)),
          ("wave", dict(scale=8.0, trained=8192, lo=1.0, hi=4.0)),
          ("ramp", dict(scale=16.0, trained=4096, lo=1.0, hi=32.0)),
          ("ramp", dict(scale=1.0, trained=2048, lo=1.0, hi=32.0))]


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("scaling,kw", SCALED)
def test_rope_freqs(L, rot, base, scaling, kw):
    f, factor = dash.rope_freqs(rot, base, scaling, **kw)
    ref, ref_factor = V.rope_freqs(rot, base, scaling, **kw)
    # a dozen operations in 64 bits on each side, each off by at most 2^-53; pow's argument is up to
    # ln(base * scale) ~ 15, which scales its own error: 64 * 2^-53 relative covers both
    assert np.abs(f.numpy() / ref - 1).max() <= 64 * 2.0 ** -53
    assert abs(factor - ref_factor) <= 2.0 ** -24 * ref_factor * 1.01   # one rounding to fp32


def test_rope_freqs_slowest_pair_of_a_raised_base(L):
    f, _ = dash.rope_freqs(128, 10000.0, "base", scale=4.0)
    g, _ = dash.rope_freqs(128, 10000.0)
    assert f[0] == 1.0 and abs(float(f[-1] * 4 / g[-1]) - 1) < 1e-13


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=2), dict(base=1.0), dict(base=float("nan")), dict(scale=0.5),
                                dict(scaling="wave", trained=0), dict(scaling="ramp", trained=64, lo=2.0, hi=1.0)])
def test_rope_freqs_refuses(L, kw):
    with pytest.raises(dash.DashError):
        dash.rope_freqs(**{**dict(rot=64, base=10000.0), **kw})


def heads(data=OK, fp32=0, n=2, sb=512, sh=128, ss=256):
    return Heads(data, fp32, n, sb, sh, ss)


FREQ = (ctypes.c_double * 64)(*[1.0 / (i + 1) for i in range(64)])


def call_rope(L, x=None, y=None, x2=None, y2=None, pos_b=0, freq=FREQ, rot=64, inter=0, factor=1.0, inverse=0, B=2, S=4, D=64):
    ref = lambda h: ctypes.byref(h) if h is not None else None  # noqa: E731
    x, y = heads() if x is None else x, heads(OK * 2) if y is None else y
    return L.dash_rope(ref(x), ref(y), ref(x2), ref(y2), None, pos_b, ctypes.cast(freq, P) if freq else None, rot, inter, factor,
                       inverse, B, S, D, None)


@pytest.mark.parametrize("kw", [
    dict(x=heads(BAD)), dict(y=heads(BAD)), dict(x=heads(None)), dict(x=heads(n=3)), dict(y=heads(n=0), x=heads(n=0)),
    dict(x=heads(sb=-512)), dict(y=heads(sh=4)), dict(y=heads(ss=0)), dict(x=heads(fp32=2)), dict(x=heads(), y=heads(sh=64)),
    dict(x=heads(), y=heads(fp32=1)), dict(x2=heads(3 * OK)), dict(y2=heads(3 * OK)), dict(rot=24), dict(rot=0), dict(rot=80),
    dict(D=96), dict(inter=2), dict(inverse=2), dict(factor=float("inf")), dict(factor=float("nan")), dict(freq=None),
    dict(freq=(ctypes.c_double * 64)(float("nan"))), dict(freq=(ctypes.c_double * 64)(1e13)), dict(B=-1), dict(S=-1),
    dict(pos_b=-1)])
def test_rope_refuses(L, kw):
    assert call_rope(L, **kw) == dash.ERR_ARG


def test_empty_calls_do_nothing(L):
    assert call_rope(L, B=0) == dash.OK and call_rope(L, S=0) == dash.OK
    assert call_write(L, T=0, k=None, v=None, slots=None) == dash.OK
    assert call_read(L, B=0) == dash.OK and call_read(L, S=0) == dash.OK
    assert call_attn(L, B=0) == dash.OK and call_attn(L, T=0, q=None, o=None) == dash.OK


def cache(k=OK, v=OK, ks=None, vs=None, typ=0, pages=4, page=16, H=2, D=64):
    return Cache(k, v, ks, vs, typ, pages, page, H, D)


BAD_CACHES = [cache(k=None), cache(v=BAD), cache(ks=OK, vs=OK), cache(typ=1), cache(typ=1, ks=OK), cache(typ=1, ks=OK, vs=BAD),
              cache(typ=2), cache(pages=0), cache(page=8), cache(page=48), cache(page=512), cache(H=0), cache(D=96),
              cache(pages=2 ** 30, H=2)]


def call_write(L, c=None, k=OK, ks=(128, 64), v=OK, vs=(128, 64), slots=OK, T=3, rope=None):
    c = cache() if c is None else c
    return L.dash_kv_write(ctypes.byref(c), k, *ks, v, *vs, slots, T, ctypes.byref(rope) if rope else None, None)


def write_rope(freq=FREQ, positions=OK, rot=64, inter=0, factor=1.0, q=OK, qs=(256, 64), q_out=2 * OK, qo=(256, 64), Hq=4):
    return WriteRope(ctypes.cast(freq, P) if freq else None, positions, rot, inter, factor, q, *qs, q_out, *qo, Hq)


@pytest.mark.parametrize("kw", [dict(c=c) for c in BAD_CACHES] + [
    dict(k=None), dict(k=BAD), dict(v=BAD), dict(ks=(-128, 64)), dict(ks=(128, 4)), dict(vs=(12, 64)), dict(slots=None),
    dict(slots=OK + 4), dict(T=-1), dict(rope=write_rope(freq=None)), dict(rope=write_rope(positions=None)),
    dict(rope=write_rope(rot=128)), dict(rope=write_rope(inter=3)), dict(rope=write_rope(q_out=None)),
    dict(rope=write_rope(q=BAD)), dict(rope=write_rope(Hq=0)), dict(rope=write_rope(qo=(0, 64))),
    dict(rope=write_rope(q_out=OK, qo=(512, 64))), dict(rope=write_rope(factor=float("nan")))])
def test_write_refuses(L, kw):
    assert call_write(L, **kw) == dash.ERR_ARG


def call_read(L, c=None, table=OK, ts=2, pages=2, lens=OK, k=OK, v=OK, strides=(4096, 2048, 64), B=2, S=32):
    c = cache() if c is None else c
    return L.dash_kv_read(ctypes.byref(c), table, ts, pages, lens, k, v, *strides, B, S, None)


@pytest.mark.parametrize("kw", [dict(c=c) for c in BAD_CACHES] + [
    dict(table=None), dict(table=BAD), dict(ts=-1), dict(pages=-1), dict(lens=None), dict(lens=BAD), dict(k=None), dict(v=BAD),
    dict(strides=(4096, 2048, 60)), dict(strides=(0, 2048, 64)), dict(strides=(4096, 2048, 0)), dict(B=-1), dict(S=-2)])
def test_read_refuses(L, kw):
    assert call_read(L, **kw) == dash.ERR_ARG


def call_attn(L, q=OK, qs=(256, 64), c=None, table=OK, ts=2, pages=2, lens=OK, cu=OK, o=OK, lse=OK, B=2, T=6, Hq=4, max_q=4,
              causal=1, window=0, ws=OK, wn=1 << 40):
    c = cache() if c is None else c
    return L.dash_attn_paged(q, *qs, ctypes.byref(c), table, ts, pages, lens, cu, o, lse, B, T, Hq, max_q, causal, window, ws, wn,
                             None)


@pytest.mark.parametrize("kw", [dict(c=c) for c in BAD_CACHES] + [
    dict(q=None), dict(q=BAD), dict(qs=(-256, 64)), dict(qs=(256, 4)), dict(table=None), dict(table=BAD), dict(ts=-2),
    dict(pages=-1), dict(lens=None), dict(lens=BAD), dict(cu=BAD), dict(o=None), dict(o=BAD), dict(lse=BAD), dict(B=-1),
    dict(T=-1), dict(Hq=3), dict(Hq=0), dict(Hq=258, c=cache(H=2)), dict(max_q=-1), dict(causal=2), dict(window=-1),
    dict(causal=0, window=5), dict(cu=None, T=5), dict(cu=None, T=12, max_q=4)])
def test_attn_refuses(L, kw):
    assert call_attn(L, **kw) == dash.ERR_ARG


def test_attn_refuses_a_small_workspace(L):
    need = dash.attn_paged_workspace(2, 2, 32, 8, 128, 1, 1 << 17)
    if need:
        assert call_attn(L, c=cache(H=8, D=128, page=16), Hq=32, T=2, max_q=1, pages=1 << 13, wn=need - 1) == dash.ERR_SCRATCH
        assert call_attn(L, c=cache(H=8, D=128, page=16), Hq=32, T=2, max_q=1, pages=1 << 13, ws=None) == dash.ERR_ARG


@pytest.mark.parametrize("a", [(-1, 1, 2, 2, 64, 1, 1), (1, -1, 2, 2, 64, 1, 1), (1, 1, 3, 2, 64, 1, 1), (1, 1, 2, 0, 64, 1, 1),
                               (1, 1, 129, 1, 64, 1, 1), (1, 1, 2, 2, 32, 1, 1), (1, 1, 2, 2, 64, -1, 1), (1, 1, 2, 2, 64, 1, -1)])
def test_workspace_refuses(L, a):
    with pytest.raises(dash.DashError):
        dash.attn_paged_workspace(*a)


def test_refuses_positions_off_their_alignment_and_outputs_past_2_30_rows(L):
    x, y = heads(), heads(OK * 2)
    assert L.dash_rope(ctypes.byref(x), ctypes.byref(y), None, None, OK + 2, 0, ctypes.cast(FREQ, P), 64, 0, 1.0, 0, 2, 4, 64,
                       None) == dash.ERR_ARG
    assert call_read(L, S=(1 << 30) + 1) == dash.ERR_ARG


@pytest.mark.parametrize("kw", [dict(qs=(0, 64)), dict(qs=(256, 0))])
def test_attn_refuses_queries_with_a_stride_of_zero(L, kw):
    assert call_attn(L, **kw) == dash.ERR_ARG


def test_status_refuses_null(L):
    assert L.dash_get_status_paged(None, None, None) == dash.ERR_ARG


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((dash.DashError, RuntimeError, AssertionError)):
        dash.rope(x, x, torch.ones(32, dtype=torch.float64))


# ---------------------------------------------------------------- the oracle itself
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_is_a_rotation_and_its_inverse(interleaved):
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 96))
    f, _ = V.rope_freqs(64, 10000.0)
    pos = np.array([0, 1, 17, 100000, 2 ** 31 - 1])
    y = V.rope(x, pos, f, 1.0, interleaved)
    assert np.allclose(V.rope(y, pos, f, 1.0, interleaved, inverse=True), x, atol=1e-12)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1)) and np.array_equal(y[0], x[0])
    # scores depend on the difference of positions alone
    a, b = V.rope(x[1], 105, f, 1.0, interleaved), V.rope(x[2], 100, f, 1.0, interleaved)
    c, d = V.rope(x[1], 5, f, 1.0, interleaved), V.rope(x[2], 0, f, 1.0, interleaved)
    assert math.isclose(a @ b, c @ d, rel_tol=1e-9)


def test_oracle_rope_gradient_by_differences():
    r = np.random.default_rng(1)
    x, g = r.standard_normal((3, 64)), r.standard_normal((3, 64))
    f, _ = V.rope_freqs(32, 100.0)
    pos = np.array([3, 50, 1000])
    grad = V.rope(g, pos, f, 1.3, True, inverse=True)
    h = 1e-6
    for i in range(64):
        e = np.zeros_like(x)
        e[:, i] = h
        num = ((V.rope(x + e, pos, f, 1.3, True) - V.rope(x - e, pos, f, 1.3, True)) * g).sum(-1) / (2 * h)
        assert np.allclose(num, grad[:, i], atol=1e-8)


def test_oracle_e4m3_grid_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = np.sort(codes[np.isfinite(codes)])
    assert np.array_equal(V.e4m3_round(codes), codes)
    mid = (codes[1:] + codes[:-1]) / 2
    for x in (mid, mid * (1 + 1e-12), mid * (1 - 1e-12)):
        ref = torch.from_numpy(x).float().to(torch.float8_e4m3fn).float().numpy() if x is mid else None
        near = V.e4m3_round(x)
        assert np.abs(near - x).max() <= np.abs(codes[None] - x[:, None]).min(1).max() + 1e-9
        if ref is not None:
            assert np.array_equal(near, ref)


def test_oracle_attend_matches_the_contiguous_oracle():
    from oracle import attention as A
    r = np.random.default_rng(2)
    S, Hq, Hkv, D = 24, 4, 2, 64
    q, k, v = (torch.from_numpy(r.standard_normal((1, h, S, D))).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    t = lambda x: x[0].transpose(0, 1).double().numpy()  # noqa: E731
    for causal, window in ((True, None), (True, 5), (False, None)):
        o, lse = A.attn_fwd(q, k, v, causal, window=window)
        for first in (0, 10):
            a, b = V.attend(t(q)[first:], t(k), t(v), first, causal, window or 0)
            assert np.allclose(a, o[0].transpose(1, 0, 2)[first:]) and np.allclose(b, lse[0].T[first:])
