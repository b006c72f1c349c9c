"""Paged attention at the edges of its protocol and its arithmetic: runs of the smallest items, weights far apart,
errors of several kernels at once, workspaces of exactly the size asked for, long contexts."""
import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from serving_helpers import DEV, check_attn, no_error, paged, randn, run_attn, same
from test_gpu_paged import CASES

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [False, True])
def test_many_items_of_one_row_tile_and_one_key_tile(D, quant):
    # Some 25 items for each SM, every one of them a single row tile (33 to 128 rows) over a single key tile: queries, keys
    # and values of two items are staged at once, and the roles that stage them run as far ahead of the products as they can.
    g = gen(60)
    B = 480
    lens = [17 + 37 * i % 112 for i in range(B)]
    n = [9 + i % 8 if i % 16 else 12 for i in range(B)]
    c = paged(g, lens, 8, D, 16, quant)
    q = randn(g, sum(n), 32, D)
    o, lse = run_attn(c, q, n)
    no_error()
    check_attn(c, q, n, o, lse)
    for _ in range(20):
        again = run_attn(c, q, n)
        no_error()
        assert same(o, again[0]) and same(lse, again[1])


def one_key_above_the_rest(c, above, q0, column):
    """Token 0 of every sequence scores `above` powers of two over the others (its key lies along the queries' first value,
    q0, which the other keys do not have); its value is zero (column None), or 64 in one column and zero in the others."""
    D, page = c.k_cache.shape[3], c.k_cache.shape[2]
    for b in range(len(c.k)):
        ln = c.k[b].shape[0]
        j = torch.arange(ln)
        p, o = c.table[b].cpu().long()[j // page].to(DEV), (j % page).to(DEV)
        k = torch.zeros(D, dtype=torch.float64)
        k[0] = above * np.log(2.0) * np.sqrt(D) / q0
        v = torch.zeros(D, dtype=torch.float64)
        if column is not None:
            v[column] = 64.0
        raw_k, raw_v = c.k_cache.view(torch.uint8), c.v_cache.view(torch.uint8)
        raw_k[p, :, o, 0] = 0
        c.k[b][:, :, 0] = 0.0
        for raw, scale, held, x in ((raw_k, c.k_scale, c.k, k), (raw_v, c.v_scale, c.v, v)):
            s = max(float(torch.tensor(float(x.abs().max()) / 448.0, dtype=torch.float32)), 2.0 ** -126)
            code = (x / s).to(torch.float32).to(torch.float8_e4m3fn)
            raw[p[0], :, o[0]] = code.view(torch.uint8).to(DEV)
            scale[p[0], :, o[0]] = s
            held[b][0] = code.double().numpy() * s


def held_to_fp16(c, q, n, o, window=None):
    """The bound of an e4m3 cache's attention.  Weights are fp16; with the largest lifted to 2^7 at least, each is off by 2^-11
    of itself or, below fp16's least normal value, by 2^-25 in units of the largest over 2^7, that is 2^-32 of the largest:
      2^-11 A                          weights
      2^-32 sum |v|                    many rows: weights below 2^-14 in fp16
      2^-32 max(P s) sum |v / s|       few rows: there the value's scale s is part of the weight
      2^-11 A + 2^-31 max |v|          many rows: values
      2^-10 A                          fp32 (see check_attn)
      2^-8 |o|                         o's own rounding to bf16"""
    o, at = o.double().cpu().numpy(), 0
    Hq, Hkv, D, page = q.shape[1], c.k_cache.shape[1], c.k_cache.shape[3], c.k_cache.shape[2]
    heads = np.arange(Hq) // (Hq // Hkv)
    for b, m in enumerate(n):
        ln, x, args = c.k[b].shape[0], q[at:at + m].double().numpy(), (c.k[b].shape[0] - m, True, window or 0)
        ro, _ = V.attend(x, c.k[b], c.v[b], *args)
        A, _ = V.attend(x, c.k[b], np.abs(c.v[b]), *args)
        j = torch.arange(ln)
        s = c.v_scale.cpu()[c.table[b].cpu().long()[j // page], :, j % page].double().numpy()      # [len, Hkv]
        few = m * (Hq // Hkv) <= 32
        if few:
            top, _ = V.attend(x, c.k[b], np.repeat(s[:, :, None], D, 2), *args)   # sum P s, at least max P s
            small = 2.0 ** -32 * top * (np.abs(c.v[b]) / s[..., None]).sum(0)[heads]
        else:
            small = 2.0 ** -32 * np.abs(c.v[b]).sum(0)[heads] + 2.0 ** -31 * np.abs(c.v[b]).max((0, 2), initial=0.0)[heads][:, None]
        bound = (2.0 ** -11 * (1 if few else 2) + 2.0 ** -10) * A + 2.0 ** -8 * np.abs(ro) + small
        d = np.abs(o[at:at + m] - ro)
        assert (d <= bound).all(), "sequence %d off by %.3g of its bound" % (b, (d / np.maximum(bound, 1e-300)).max())
        at += m


@pytest.mark.parametrize("name", ["one_of_1000", "decode_ragged", "decode_window", "decode_wide_group", "two_tokens", "verify", "chunk",
                                  "chunk_ragged", "chunk_window", "chunk_odd_group", "mixed", "mixed_window", "group_128"])
def test_e4m3_caches_are_held_to_their_own_bound(name):
    Hq, Hkv, D, page, lens, n, window, pad = CASES[name]
    g = gen(65)
    c = paged(g, lens, Hkv, D, page, True)
    q = randn(g, sum(n) + pad, Hq, D)
    o, _ = run_attn(c, q, n, window=window)
    no_error()
    held_to_fp16(c, q, n, o, window)


@pytest.mark.parametrize("n", [[1, 1], [5, 8], [9, 40], [33, 1]])   # four heads each: up to 8 tokens are few rows
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("above,column", [(16, None), (20, None), (24, None), (26, None), (16, 3), (20, 3)])
def test_weights_far_below_the_largest(n, D, above, column):
    # The first key takes nearly all of the weight and its value is zero (or large in one column alone), so the other keys, each
    # 2^-above of it, are the whole output: held to the bound of held_to_fp16, whose fp32 part holds here too (scores have
    # absolute sums below 12 sqrt(D); the first key's score is one product, exact).
    g = gen(61)
    c = paged(g, [1500, 700], 2, D, 16, True)
    for b in range(2):   # values around one: their sum does not cancel
        ln, page = c.k[b].shape[0], 16
        j = torch.arange(ln)
        p, o = c.table[b].cpu().long()[j // page].to(DEV), (j % page).to(DEV)
        x = 1.0 + 0.25 * torch.randn(ln, 2, D, generator=g)
        s = x.abs().amax(-1) / 448.0
        code = (x / s[..., None]).to(torch.float8_e4m3fn)
        c.v_cache.view(torch.uint8)[p, :, o] = code.view(torch.uint8).to(DEV)
        c.v_scale[p, :, o] = s.to(DEV)
        c.v[b][:] = code.double().numpy() * s.double().numpy()[..., None]
    one_key_above_the_rest(c, above, 8.0, column)
    q = randn(g, sum(n), 8, D)
    q[:, :, 0] = 8.0
    o, lse = run_attn(c, q, n)
    no_error()
    held_to_fp16(c, q, n, o)
    at = 0
    for b, m in enumerate(n):
        _, rl = V.attend(q[at:at + m].double().numpy(), c.k[b], c.v[b], c.k[b].shape[0] - m)
        got = lse[at:at + m].cpu().double().numpy()
        assert (np.abs(got - rl) <= 2.0 ** -12 + 2.0 ** -20 * np.abs(rl)).all()
        at += m


def test_errors_of_several_kernels_are_all_reported():
    # a slot past the cache (writer), a bad page of a sequence of few rows and one of a sequence of many: three reports,
    # whatever their order in time, each once
    g = gen(62)
    c = paged(g, [300, 200], 2, 64, 16, False)
    q = randn(g, 61, 4, 64)
    good, bad = c.table.clone(), c.k_cache.shape[0] + 9
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    slot = torch.tensor([c.k_cache.shape[0] * 16 + 5], dtype=torch.int64, device=DEV)
    for order in ((0, 1, 2), (2, 1, 0), (1, 2, 0)):
        for what in order:
            c.table = good.clone()
            if what == 0:
                dash.kv_write(x, x, c.k_cache, c.v_cache, slot)
            else:   # sequence 0 has 60 new tokens (many rows), sequence 1 one (few)
                c.table[2 - what, 2] = bad + what
                run_attn(c, q, [60, 1])
        c.table = good
        got = [dash.get_status_paged() for _ in range(3)]
        assert [code for code, _ in got] == [dash.ERR_PAGE] * 3
        assert got[0][1] == [1, 0, int(slot), c.k_cache.shape[0] * 16]
        assert got[1][1] == [3, 1, bad + 1, c.k_cache.shape[0]] and got[2][1] == [3, 0, bad + 2, c.k_cache.shape[0]]
        no_error()


@pytest.mark.parametrize("n,lens", [([1], [40000]), ([1] * 5, [9000] * 5), ([5, 5], [6000, 6000]), ([30, 1, 7], [5000, 9000, 7000]),
                                    ([200], [8000])])
@pytest.mark.parametrize("quant", [False, True])
def test_a_workspace_of_exactly_the_size_asked_for(n, lens, quant):
    # every cut into key ranges lies inside it: the bytes behind stay as they are, and the results are those with a large one
    Hq, Hkv, D, page = 8, 2, 64, 16
    g = gen(63)
    c = paged(g, lens, Hkv, D, page, quant)
    q = randn(g, sum(n), Hq, D)
    need = dash.attn_paged_workspace(len(n), sum(n), Hq, Hkv, D, max(n), c.table.shape[1] * page)
    assert need > 0
    large = torch.zeros(2 * need + (1 << 20), dtype=torch.uint8, device=DEV)
    o, lse = run_attn(c, q, n, workspace=large)
    no_error()
    buf = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device=DEV)
    o2, lse2 = run_attn(c, q, n, workspace=buf[:need])
    no_error()
    assert same(o, o2) and same(lse, lse2)
    assert bool((buf[need:] == 0xa5).all())
    check_attn(c, q, n, o, lse)


LONG = {
    # name: (Hq, Hkv, D, page, lens, new tokens, window)
    # few rows: a row in more than 48 key ranges (joined by a block), with and without a short sequence beside it
    "many_ranges": (4, 1, 128, 32, [41003], [1], None),
    "many_ranges_beside_one": (8, 2, 64, 16, [40001, 7], [1, 1], None),
    "many_ranges_drafts": (4, 1, 64, 64, [39990, 30011], [4, 2], None),
    # ranges of more than 32 pages, through which a group's producer follows the table
    "long_ranges": (8, 8, 128, 16, [25013], [1], None),
    "long_ranges_drafts": (16, 8, 128, 16, [25013, 600], [3, 1], None),
    "long_ranges_batch": (32, 32, 64, 16, [9001, 8190, 12345], [1, 1, 1], None),
    # a window that begins inside a page, a stage and a range
    "window": (8, 2, 128, 16, [45678, 20000], [1, 2], 30007),
    "window_few_heads": (2, 1, 64, 32, [50021], [1], 44444),
    # many rows: key ranges beside few-rows ones, and more than 32 pages to a range
    "chunk": (4, 1, 128, 16, [20011, 33000], [50, 1], None),
    "chunk_window": (8, 4, 64, 16, [15001], [70], 9999),
}


@pytest.mark.parametrize("name", list(LONG))
@pytest.mark.parametrize("quant", [False, True])
def test_long_contexts(name, quant):
    Hq, Hkv, D, page, lens, n, window = LONG[name]
    g = gen(64)
    c = paged(g, lens, Hkv, D, page, quant)
    q = randn(g, sum(n), Hq, D)
    o, lse = run_attn(c, q, n, window=window)
    no_error()
    check_attn(c, q, n, o, lse, window=window)
    if window is None:
        o, lse = run_attn(c, q, n, causal=False)
        no_error()
        check_attn(c, q, n, o, lse, causal=False)
