"""The cache of 4 bits without a GPU: its rounding against a search of the grid, and every refusal that needs no device."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from cache4_helpers import quantised4, values4

P, I, Z, H = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int16


class Cache(ctypes.Structure):       # dash_kv_cache
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("type", I), ("num_pages", I), ("page_size", I),
                ("Hkv", I), ("D", I), ("k_exp", H), ("v_exp", H)]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dash.lib()


def test_the_bindings_layout_is_the_struct():
    assert dash._CACHE_EXP.size == dash._CACHE.size == ctypes.sizeof(Cache)
    values = list(range(1, 10)) + [-3, 5]
    got = Cache.from_buffer_copy(dash._CACHE_EXP.pack(*values))
    assert [getattr(got, f) for f, _ in Cache._fields_] == values
    plain = Cache.from_buffer_copy(dash._CACHE.pack(*values[:9]))
    assert [getattr(plain, f) for f, _ in Cache._fields_] == values[:9] + [0, 0]


def test_rounding_by_searching_the_grid():
    """Every tie and its neighbours, and random values: the nearest grid value, ties to the even code; both plain forms."""
    grid = V.E2M1
    y = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, np.random.default_rng(0).uniform(0, 6, 1000)])
    y = np.concatenate([y, -y, [6.0] * ((-2 * y.size) % 16)])
    y = y.reshape(-1, 16)
    y[:, 0] = 6.0                                        # the block's largest: a scale of one
    y = torch.tensor(y, dtype=torch.float32).double().numpy()
    best = np.empty_like(y)
    for at in np.ndindex(*y.shape):
        d = np.abs(grid - abs(y[at]))
        near = np.flatnonzero(d == d.min())
        best[at] = np.copysign(grid[near[near % 2 == 0][0] if near.size > 1 else near[0]], y[at])
    code, scale = V.quantise4(y, 0)
    assert (scale == 1.0).all() and np.array_equal(code, best)
    raw, s = quantised4(torch.tensor(y, dtype=torch.float32), 0)
    assert np.array_equal(values4(raw, s, 0).numpy(), best)


@pytest.mark.parametrize("exp", [-5, 0, 3])
def test_both_plain_forms_agree(exp):
    x = torch.randn(200, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** 14
    x[2] *= 2.0 ** -14
    raw, s = quantised4(x, exp)
    code, scale = V.quantise4(x.double().numpy(), exp)
    assert np.array_equal(values4(raw, s, exp).numpy(), code * np.repeat(scale, 16, -1))
    assert np.array_equal(s.float().double().numpy() * 2.0 ** exp, scale)


OK, BAD = 4096, 4098   # an aligned and a misaligned address, never dereferenced


def cache(k=OK, v=OK, ks=OK, vs=OK, typ=2, pages=4, page=16, Hkv=2, D=64, ke=0, ve=0):
    return Cache(k, v, ks, vs, typ, pages, page, Hkv, D, ke, ve)


BAD_CACHES = [cache(k=None), cache(v=BAD), cache(ks=None), cache(vs=None), cache(ks=BAD), cache(vs=BAD), cache(typ=3), cache(pages=0),
              cache(page=8), cache(page=48), cache(page=512), cache(Hkv=0), cache(D=96), cache(D=32), cache(ke=65), cache(ke=-65),
              cache(ve=65), cache(ve=-65), cache(pages=2 ** 30)]


@pytest.mark.parametrize("c", BAD_CACHES)
def test_a_bad_cache_is_refused_by_every_call(L, c):
    r = ctypes.byref(c)
    assert L.dash_kv_write(r, OK, 128, 64, OK, 128, 64, OK, 3, None, None) == dash.ERR_ARG
    assert L.dash_kv_read(r, OK, 8, 4, OK, OK, OK, 4096, 1024, 64, 2, 4, None) == dash.ERR_ARG
    assert L.dash_attn_paged(OK, 256, 64, r, OK, 8, 4, OK, OK, OK, None, 2, 3, 4, 2, 1, 0, OK, 1 << 30, None) == dash.ERR_ARG


def test_an_empty_call_does_nothing(L):
    r = ctypes.byref(cache())
    assert L.dash_kv_write(r, None, 128, 64, None, 128, 64, None, 0, None, None) == dash.OK
    assert L.dash_kv_read(r, None, 8, 4, None, None, None, 4096, 1024, 64, 0, 4, None) == dash.OK
    assert L.dash_attn_paged(None, 256, 64, r, None, 8, 4, None, None, None, None, 0, 0, 4, 2, 1, 0, None, 0, None) == dash.OK


@pytest.mark.parametrize("exps", [dict(k_exp=-3), dict(v_exp=2), dict(k_exp=1, v_exp=1)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_exponents_belong_to_caches_of_4_bits(L, monkeypatch, kind, exps):
    monkeypatch.setattr(dash, "_device_stream", lambda stream, what: (-1, 0))   # (CPU tensors stand for the device's)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    s = torch.zeros(4, 2, 16)
    kw = dict(exps) if kind == "bf16" else dict(exps, k_scale=s, v_scale=s)
    x, out = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: dash.kv_write(x, x, c, c, torch.zeros(3, dtype=torch.int64), **kw),
                 lambda: dash.kv_read(c, c, table, lens, out, out, **kw),
                 lambda: dash.attn_paged(x, c, c, table, lens, x, workspace=torch.zeros(16, dtype=torch.uint8), **kw)):
        with pytest.raises(dash.DashError, match="k_exp"):
            call()
