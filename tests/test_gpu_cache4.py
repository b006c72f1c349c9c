"""A paged cache of 4 bits on the GPU: written, read back and attended to, against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from cache4_helpers import check_attn4, paged4, quantised4, values4
from serving_helpers import DEV, E4M3, no_error, randn, rope_bound, run_attn, same

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------------------------------------------- writing
WRITES = {
    # name: (T, Hq, Hkv, D, page, rot, interleaved)
    "one_token": (1, 2, 1, 64, 16, 64, False),
    "halves": (67, 8, 2, 128, 16, 128, False),
    "pairs": (130, 4, 4, 64, 64, 64, True),
    "quarter": (33, 6, 2, 64, 32, 16, True),
    "odd_sixteenths": (50, 3, 3, 128, 128, 48, False),
    "odd_sixteenths_pairs": (19, 4, 1, 128, 256, 80, True),
    "many_heads": (700, 28, 4, 128, 16, 112, False),
}


def empty4(N, Hkv, page, D):
    return [torch.full((N, Hkv, page, D // w), 3, dtype=torch.uint8, device=DEV) for w in (2, 2, 16, 16)]


def written(name, rotate, seed=3, special=False):
    T, Hq, Hkv, D, page, rot, pairs = WRITES[name]
    g = gen(seed)
    qkv = randn(g, T, Hq + 2 * Hkv, D)
    if special:   # zeros, far magnitudes, and what is not finite
        qkv[0, Hq:, :16] = 0
        qkv[0, Hq:, 16:32] = 2.0 ** -20
        qkv[0, Hq:, 32:48] *= 2.0 ** 20
        qkv[T // 2, Hq:, 3] = float("inf")
        qkv[T // 2, Hq:, 63] = float("nan")
        qkv[T - 1, Hq:, 17] = float("-inf")
    N = -(-T // page) + 2
    slots = (torch.randperm(N, generator=g)[:, None] * page + torch.arange(page)).flatten()[:T].clone()
    if T > 10:
        slots[5] = -1
        slots[T - 1] = -9
    kc, vc, ks, vs = empty4(N, Hkv, page, D)
    d = qkv.to(DEV)
    q, k, v = d.split([Hq, Hkv, Hkv], dim=1)
    out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    freqs, factor = dash.rope_freqs(rot)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    turn = dict(inv_freq=freqs, positions=pos.to(DEV), interleaved=pairs, factor=factor, q=q, q_out=out) if rotate else {}
    dash.kv_write(k, v, kc, vc, slots.to(DEV), k_scale=ks.view(E4M3), v_scale=vs.view(E4M3), k_exp=-3, v_exp=2, **turn)
    no_error()
    return qkv, slots, pos, freqs, factor, (kc, vc, ks, vs), out


@pytest.mark.parametrize("name", list(WRITES))
@pytest.mark.parametrize("special", [False, True])
def test_write_without_rotation(name, special):
    """Byte for byte what the definition gives in fp32; every other cell keeps its bytes."""
    T, Hq, Hkv, D, page, _, _ = WRITES[name]
    qkv, slots, _, _, _, got, _ = written(name, False, special=special)
    ok = slots >= 0
    p, o = slots[ok] // page, slots[ok] % page
    for x, exp, codes, scales in ((qkv[:, Hq:Hq + Hkv], -3, got[0], got[2]), (qkv[:, Hq + Hkv:], 2, got[1], got[3])):
        c, s = quantised4(x[ok], exp)
        wc, ws = torch.full(codes.shape, 3, dtype=torch.uint8), torch.full(scales.shape, 3, dtype=torch.uint8)
        wc[p, :, o], ws[p, :, o] = c, s.view(torch.uint8)
        dead = (ws == 0x7f).repeat_interleave(8, -1)   # a NaN scale says it all: its codes may be anything
        assert torch.equal(scales.cpu(), ws)
        assert torch.equal(codes.cpu()[~dead], wc[~dead])


@pytest.mark.parametrize("name", list(WRITES))
def test_write_with_rotation(name):
    """A rotated key is off by fp32's rounding (rope_bound's first term), so that its code or its block's scale is another
    where it lies that near to a border: a share of a few 2^-19 of each other code's step, so one value in a thousand is
    far more than can come of it; such a value is off by a step (of a third at most) of its block's largest."""
    T, Hq, Hkv, D, page, rot, pairs = WRITES[name]
    qkv, slots, pos, freqs, factor, got, out = written(name, True)
    x = qkv.double().numpy()
    turned = V.rope(x[:, :Hq + Hkv], pos.numpy()[:, None], freqs.numpy(), factor, pairs)
    ref = turned[:, :Hq]
    assert (np.abs(out.float().cpu().double().numpy() - ref) <= rope_bound(x[:, :Hq], freqs.numpy(), factor, pairs, True, ref)).all()
    ok = (slots >= 0).numpy()
    p, o = slots[slots >= 0] // page, slots[slots >= 0] % page
    for y, exp, codes, scales in ((turned[ok, Hq:], -3, got[0], got[2]), (x[ok, Hq + Hkv:], 2, got[1], got[3])):
        held = values4(codes.cpu()[p, :, o], scales.cpu()[p, :, o].view(E4M3), exp).numpy()
        code, scale = V.quantise4(y, exp)
        want = code * np.repeat(scale, 16, -1)
        d = np.abs(held - want)
        top = np.repeat(np.abs(y).reshape(y.shape[:-1] + (-1, 16)).max(-1), 16, -1)
        assert (d > 0).mean() <= 1e-3
        assert (d <= 0.375 * top).all()


def test_write_reports_a_slot_past_the_cache():
    kc, vc, ks, vs = empty4(2, 1, 16, 64)
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    dash.kv_write(x, x, kc, vc, torch.tensor([1, 32, 31], device=DEV), k_scale=ks.view(E4M3), v_scale=vs.view(E4M3))
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info == [1, 1, 32, 32]
    assert (kc[0, 0, 1] != 3).all() and (kc[1, 0, 15] != 3).all() and int((kc != 3).sum()) == 64


# ---------------------------------------------------------------------------------------------------------------- reading
@pytest.mark.parametrize("D,Hkv,page,lens,S", [(64, 2, 16, [1, 0, 33], 40), (128, 4, 64, [300, 129], 300), (128, 1, 256, [700], 600),
                                               (64, 3, 128, [5, 6, 7, 1000], 1000)])
def test_read(D, Hkv, page, lens, S):
    c = paged4(gen(4), lens, Hkv, D, page, exps=(5, -7))
    k, v = (torch.full((len(lens), S, Hkv, D), 9.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2) for _ in range(2))
    dash.kv_read(c.k_cache, c.v_cache, c.table, c.lens, k, v, **c.kw)
    no_error()
    for got, ref in ((k, c.k), (v, c.v)):
        got = got.float().cpu().double().numpy()
        for b, n in enumerate(lens):
            m = min(n, S)
            # (two bits of a code, four of a scale, a power of two: bf16 holds it)
            assert np.array_equal(got[b, :, :m], ref[b][:m].transpose(1, 0, 2)) and (got[b, :, m:] == 9.0).all()


def test_a_block_that_is_not_finite_reads_back_as_nan():
    D, page = 64, 16
    kc, vc, ks, vs = empty4(1, 1, page, D)
    kw = dict(k_scale=ks.view(E4M3), v_scale=vs.view(E4M3))
    x = torch.ones(2, 1, D, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 20] = float("nan")
    x[1, 0, 40] = float("-inf")
    dash.kv_write(x, x, kc, vc, torch.tensor([0, 1], device=DEV), **kw)
    k, v = (torch.zeros(1, 1, 2, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dash.kv_read(kc, vc, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV), k, v, **kw)
    no_error()
    want = torch.full((2, D), 6 * 11 / 64)   # 1 / 6 rounds to the scale 11 / 64, 1 over it to the code of 6
    want[0, 16:32] = want[1, 32:48] = float("nan")
    for t in (k, v):
        assert torch.equal(torch.nan_to_num(t[0, 0].float().cpu(), 5.0), torch.nan_to_num(want, 5.0))


# -------------------------------------------------------------------------------------------------------------- attention
CASES = {
    # name: (Hq, Hkv, D, page, lens, new tokens, window, padding rows)
    "one_token": (2, 2, 64, 16, [1], [1], None, 0),
    "one_of_1000": (32, 8, 128, 16, [1000], [1], None, 0),
    "decode_ragged": (32, 8, 128, 64, [1, 17, 300, 129, 1025, 64], [1] * 6, None, 3),
    "decode_mha": (4, 4, 128, 128, [127, 128, 129, 2049], [1] * 4, None, 0),
    "decode_wide_group": (64, 2, 64, 32, [70, 700], [1, 1], None, 1),
    "decode_odd_group": (14, 2, 128, 16, [333, 34], [1, 1], None, 0),
    "decode_empty": (8, 2, 128, 16, [0, 40, 0], [1, 1, 1], None, 0),
    "decode_window": (8, 2, 64, 16, [5, 100, 1500], [1, 1, 1], 37, 0),
    "decode_d64": (8, 1, 64, 256, [2500, 3], [1, 1], None, 0),
    "two_tokens": (32, 8, 128, 16, [2, 515], [2, 2], None, 0),
    "verify": (32, 8, 128, 32, [700, 5, 260], [5, 5, 5], None, 2),
    "verify_small_group": (6, 2, 64, 16, [130, 512], [4, 3], None, 0),
    "rows_16_to_33": (8, 2, 128, 16, [400, 300, 290, 500], [4, 5, 8, 9], None, 0),
    "rows_16_to_33_d64": (8, 2, 64, 32, [400, 300, 290, 500], [4, 5, 8, 9], 200, 0),
    "chunk": (8, 2, 128, 64, [400], [200], None, 0),
    "chunk_ragged": (4, 4, 128, 16, [130, 900, 77], [130, 65, 1], None, 5),
    "chunk_odd_group": (14, 2, 64, 128, [640], [150], None, 0),
    "chunk_window": (8, 2, 128, 16, [700, 300], [150, 300], 100, 0),
    "chunk_window_tiny": (4, 2, 64, 16, [500], [300], 1, 0),
    "chunk_more_new_than_cached": (4, 2, 64, 16, [20, 0], [50, 3], None, 0),
    "chunk_long": (4, 1, 128, 32, [5000], [70], None, 0),
    "mixed": (16, 4, 64, 16, [1300, 1, 500, 64, 0], [1, 1, 260, 0, 1], None, 4),
    "mixed_window": (8, 8, 128, 32, [900, 800, 33], [1, 140, 33], 300, 0),
    # several items for every SM, and mixtures of one and two row tiles
    "decode_many": (16, 8, 64, 16, [37 * i % 900 + 1 for i in range(70)], [1] * 70, None, 0),
    "verify_many": (32, 8, 128, 32, [301 * i % 1900 + 6 for i in range(40)], [5] * 40, None, 0),
    "verify_many_window": (32, 8, 64, 16, [301 * i % 1900 + 6 for i in range(40)], [6] * 40, 500, 0),
    # small pages in batches that fill the GPU, with windows that begin inside a page
    "decode_many_pages_16": (16, 8, 128, 16, [53 * i % 1700 + 1 for i in range(40)], [1] * 40, None, 0),
    "decode_many_pages_32": (16, 8, 64, 32, [53 * i % 1700 + 1 for i in range(40)], [1] * 40, 333, 0),
    "decode_many_pages_16_window": (32, 4, 128, 16, [71 * i % 900 + 2 for i in range(50)], [2] * 50, 77, 2),
    "chunk_pages_16": (8, 8, 128, 16, [333, 1000, 20], [100, 333, 20], 250, 0),
    "chunk_pages_32": (8, 2, 64, 32, [333, 1000, 20], [100, 333, 20], None, 0),
    "chunk_many": (8, 8, 128, 64, [211 * i % 700 + 300 for i in range(30)], [17 * i % 300 + 17 for i in range(30)], None, 3),
    "group_128": (128, 1, 64, 16, [90, 300], [1, 3], None, 0),
}


def inputs(name, seed=1, **kw):
    Hq, Hkv, D, page, lens, n, window, pad = CASES[name]
    g = gen(seed)
    c = paged4(g, lens, Hkv, D, page, **kw)
    return c, randn(g, sum(n) + pad, Hq, D), n, window


@pytest.mark.parametrize("name", list(CASES))
def test_attention_against_the_oracle(name):
    c, q, n, window = inputs(name)
    o, lse = run_attn(c, q, n, window=window)
    no_error()
    check_attn4(c, q, n, o, lse, window=window)


@pytest.mark.parametrize("name", ["decode_ragged", "verify", "chunk_ragged", "mixed", "rows_16_to_33"])
def test_full_mask(name):
    c, q, n, _ = inputs(name, seed=2)
    o, lse = run_attn(c, q, n, causal=False)
    no_error()
    check_attn4(c, q, n, o, lse, causal=False)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_every_page_size(page, D):
    g = gen(3)
    c = paged4(g, [page * 2 + 3, 300, 1], 2, D, page)
    for n in ([1, 1, 1], [40, 33, 1]):
        q = randn(g, sum(n), 8, D)
        o, lse = run_attn(c, q, n)
        no_error()
        check_attn4(c, q, n, o, lse)


@pytest.mark.parametrize("sigma,exps", [(1.0, (0, 0)), (300.0, (0, 3)), (1e-3, (-12, -12)), (1.0, (-8, 7))])
@pytest.mark.parametrize("n", [1, 40])
def test_exponents_and_far_magnitudes(sigma, exps, n):
    """Values near the ends of what the scales hold, saturated ones among them (exponents that do not suit the data)."""
    g = gen(7)
    c = paged4(g, [500, 90], 2, 128, 16, sigma=sigma, exps=exps)
    q = (randn(g, 2 * n, 8, 128).float() / max(sigma, 1.0)).to(torch.bfloat16)
    o, lse = run_attn(c, q, [n, n])
    no_error()
    check_attn4(c, q, [n, n], o, lse)


@pytest.mark.parametrize("name", ["decode_ragged", "verify_many", "chunk_many", "mixed"])
def test_the_same_bits_in_any_batch_and_run(name):
    c, q, n, window = inputs(name, seed=5)
    o, lse = run_attn(c, q, n, window=window)
    again, lse2 = run_attn(c, q, n, window=window)
    assert same(o, again) and same(lse, lse2)
    at = np.concatenate([[0], np.cumsum(n)])
    for b in range(0, len(n), max(1, len(n) // 4)):
        rows = slice(int(at[b]), int(at[b + 1]))
        if n[b] == 0:
            continue
        one = type(c)([c.k[b]], [c.v[b]], c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table[b:b + 1].contiguous(), c.lens[b:b + 1].contiguous(), c.kw)
        oo, ol = run_attn(one, q[rows], [n[b]], window=window)
        assert same(oo, o[rows]) and same(ol, lse[rows])


# batches whose sequences have more than 8 rows: products of two and three row tiles over each key
TILES = {
    # name: (Hq, Hkv, D, page, most new tokens, window, causal)
    "two_of_64": (16, 4, 64, 16, 4, None, True),
    "two_of_128": (16, 4, 128, 32, 3, None, True),
    "two_wide_group": (64, 4, 128, 64, 1, None, True),
    "three_of_64": (16, 4, 64, 64, 5, 300, True),
    "three_of_128": (16, 4, 128, 16, 6, None, True),
    "three_odd_group": (28, 4, 128, 128, 3, 70, True),
    "three_odd_group_64": (20, 4, 64, 32, 4, 1, True),
    "two_twice_of_64": (16, 4, 64, 128, 8, 129, True),
    "two_twice_of_128": (16, 4, 128, 16, 7, None, True),
    "two_twice_wide_group": (128, 4, 64, 16, 1, 500, True),
    "three_full": (16, 4, 128, 64, 5, None, False),
    "two_full": (16, 4, 64, 64, 4, None, False),
}


def tile_inputs(name, seed=1):
    """41 sequences of 0 to `most` new tokens; some without keys, some with fewer keys than new tokens, two long ones."""
    Hq, Hkv, D, page, most, window, causal = TILES[name]
    g = gen(seed)
    lens = [149 * i % 700 for i in range(38)] + [2, 4100, 6000]
    n = [most - (i % 3 if most > 2 else 0) for i in range(41)]
    lens[7], n[11] = 0, 0
    c = paged4(g, lens, Hkv, D, page)
    return c, randn(g, sum(n) + 3, Hq, D), n, window, causal


@pytest.mark.parametrize("name", list(TILES))
def test_row_tiles_against_the_oracle(name):
    c, q, n, window, causal = tile_inputs(name)
    o, lse = run_attn(c, q, n, window=window, causal=causal)
    no_error()
    check_attn4(c, q, n, o, lse, window=window, causal=causal)


@pytest.mark.parametrize("name", list(TILES))
def test_row_tiles_give_the_same_bits_as_single_ones(name):
    """A sequence alone (single row tiles), in the batch, and in a step that prefills another sequence, too."""
    c, q, n, window, causal = tile_inputs(name, seed=6)
    o, lse = run_attn(c, q, n, window=window, causal=causal)
    at = np.concatenate([[0], np.cumsum(n)])
    for b in (0, 5, 7, 13, 38, 39, 40):
        rows = slice(int(at[b]), int(at[b + 1]))
        one = type(c)([c.k[b]], [c.v[b]], c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table[b:b + 1].contiguous(), c.lens[b:b + 1].contiguous(), c.kw)
        oo, ol = run_attn(one, q[rows], [n[b]], window=window, causal=causal)
        assert same(oo, o[rows]) and same(ol, lse[rows])
        two = type(c)([c.k[b], c.k[3]], [c.v[b], c.v[3]], c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table[[b, 3]].contiguous(),
                      c.lens[[b, 3]].contiguous(), c.kw)
        g = gen(8)
        oo, ol = run_attn(two, torch.cat([q[rows], randn(g, 40, q.shape[1], q.shape[2])]), [n[b], 40], window=window, causal=causal)
        assert same(oo[:n[b]], o[rows]) and same(ol[:n[b]], lse[rows])
    no_error()


@pytest.mark.parametrize("name", ["two_of_64", "two_of_128", "three_of_64", "three_of_128", "two_twice_of_128"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_row_tiles_of_queries_that_are_not_finite(name, bad):
    c, q, n, window, causal = tile_inputs(name, seed=7)
    want, _ = run_attn(c, q, n, window=window)
    at = [0, sum(n[:6]), sum(n[:41]) - 1]   # a long sequence's last token among them
    for x, t in enumerate(at):
        q[t, 5 * x, 3] = bad
    o, lse = run_attn(c, q, n, window=window)
    no_error()
    keep = torch.ones(q.shape[0], q.shape[1], dtype=torch.bool)
    for x, t in enumerate(at):
        keep[t, 5 * x] = False
    assert same(o[keep.to(DEV)], want[keep.to(DEV)])
    assert torch.isnan(o[at[2], 10]).all() and torch.isnan(lse[at[2], 10])


def test_a_key_far_above_the_others():
    """One key some 2^20 above the rest, with a small value: the others' weights have to keep their bits."""
    Hkv, D, page, L = 1, 64, 16, 300
    for n in (1, 40):
        g = gen(9)
        c = paged4(g, [L], Hkv, D, page, exps=(0, 0))
        codes, scales = c.k_cache.cpu(), c.k_scale.cpu().view(torch.uint8)
        vc = c.v_cache.cpu()
        p = int(c.table[0, 0])
        codes[p, 0, 0] = 0x22                       # all ones
        scales[p, 0, 0] = torch.tensor([2.0]).to(E4M3).view(torch.uint8)
        vc[p, 0, 0] = 0                             # its value: zero
        c.k_cache, c.k_scale, c.v_cache = codes.to(DEV), scales.view(E4M3).to(DEV), vc.to(DEV)
        c.kw.update(k_scale=c.k_scale)
        c.k[0][0], c.v[0][0] = 2.0, 0.0
        q = torch.full((n, 2, D), 0.875).to(torch.bfloat16)   # scores of 14 where the others are near zero
        o, lse = run_attn(c, q, [n])
        no_error()
        check_attn4(c, q, [n], o, lse)


def test_pages_out_of_range_are_reported_and_other_sequences_untouched():
    c, q, n, _ = inputs("decode_ragged")
    c.table[2, 1] = 10 ** 6
    o, lse = run_attn(c, q, n)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info[:3] == [3, 2, 10 ** 6]
    for b in (0, 1, 3, 4, 5):
        one = type(c)([c.k[b]], [c.v[b]], c.k_cache, c.v_cache, None, None, c.table[b:b + 1].contiguous(), c.lens[b:b + 1].contiguous(), c.kw)
        oo, ol = run_attn(one, q[b:b + 1], [1])
        assert same(oo, o[b:b + 1]) and same(ol, lse[b:b + 1])
    no_error()


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_zero_and_least_exponents(n, D):
    """Scores' scales far below the least normal number: masked keys stay masked, every seen one weighs the same."""
    g = gen(11)
    c = paged4(g, [200, 77], 2, D, 16, exps=(-64, 0))
    q = randn(g, 2 * n, 8, D)
    q[0] = 0
    q[n:, 3] = 2.0 ** -120
    o, lse = run_attn(c, q, [n, n])
    no_error()
    check_attn4(c, q, [n, n], o, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_that_are_not_finite_give_nan_in_their_rows_alone(bad, n, D):
    g = gen(12)
    c = paged4(g, [300], 2, D, 16)
    q = randn(g, n, 8, D)
    want, _ = run_attn(c, q, [n])
    q[n - 1, 5, 7] = bad
    o, lse = run_attn(c, q, [n])
    no_error()
    assert torch.isnan(o[n - 1, 5]).all() and torch.isnan(lse[n - 1, 5])
    keep = torch.ones(n, 8, dtype=torch.bool)
    keep[n - 1, 5] = False
    assert same(o[keep.to(DEV)], want[keep.to(DEV)])


@pytest.mark.parametrize("D", [64, 128])
def test_strided_queries_and_packed_types(D):
    """Queries inside a wider projection, caches as pairs of 4-bit floats."""
    g = gen(13)
    c = paged4(g, [90, 400], 2, D, 32)
    wide = randn(g, 7, 12, D).to(DEV)
    q = wide[:, 2:10]
    n = [3, 4]
    o, lse = run_attn(c, q, n)
    check_attn4(c, q.cpu().contiguous(), n, o, lse)
    if hasattr(torch, "float4_e2m1fn_x2"):
        packed = type(c)(c.k, c.v, c.k_cache.view(torch.float4_e2m1fn_x2), c.v_cache.view(torch.float4_e2m1fn_x2), None, None, c.table, c.lens, c.kw)
        o2, lse2 = run_attn(packed, q, n)
        assert same(o, o2) and same(lse, lse2)
    no_error()


def test_refusals_of_the_binding():
    c = paged4(gen(14), [40], 2, 64, 16)
    o = torch.empty(1, 8, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros_like(o)
    good = dict(c.kw)
    for kw in (dict(k_scale=None), dict(v_scale=c.v_scale.view(torch.uint8)), dict(k_scale=c.k_scale[..., :2]), dict(k_exp=65), dict(v_exp=-65),
               dict(k_scale=torch.zeros(c.k_cache.shape[:3], device=DEV))):
        with pytest.raises(dash.DashError):
            dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, **{**good, **kw})
    with pytest.raises(dash.DashError):
        dash.attn_paged(q, c.k_cache, c.v_cache.view(torch.int8), c.table, c.lens, o, **good)
    with pytest.raises(dash.DashError):   # 32 bytes are 64 values: the queries have as many
        dash.attn_paged(q[..., :32], c.k_cache, c.v_cache, c.table, c.lens, o, **good)
    with pytest.raises(dash.DashError):
        dash.kv_read(c.k_cache, c.v_cache, c.table, c.lens, o[None], o[None], **good)


def test_captured_and_on_another_stream():
    c, q, n, window = inputs("mixed", seed=15)
    want, wl = run_attn(c, q, n, window=window)
    q = q.to(DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    outs = [(torch.full_like(want, 77.0), torch.full_like(wl, 77.0)) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    for g, (o, l) in zip(graphs, outs):
        with torch.cuda.graph(g):
            dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=max(n), lse=l, window=window, **c.kw)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, g in zip(streams, graphs):   # two replays at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, l in outs:
        assert same(o, want) and same(l, wl)
    no_error()


@pytest.mark.parametrize("D", [64, 128])
def test_zeros_keep_their_sign(D):
    """Byte for byte the definition's: -0 beside other values, beside zeros alone, and as what a tiny value becomes."""
    x = torch.zeros(3, 1, D)
    x[0, 0, ::3] = -0.0
    x[0, 0, 1::4] = 1.5
    x[1] = -0.0
    x[2] = -2.0 ** -120
    x = x.to(torch.bfloat16)
    kc, vc, ks, vs = empty4(1, 1, 16, D)
    dash.kv_write(x.to(DEV), x.neg().to(DEV), kc, vc, torch.arange(3, device=DEV), k_scale=ks.view(E4M3), v_scale=vs.view(E4M3), k_exp=-3, v_exp=5)
    no_error()
    for y, exp, codes, scales in ((x, -3, kc, ks), (x.neg(), 5, vc, vs)):
        c, s = quantised4(y, exp)
        assert torch.equal(scales.cpu()[0, 0, :3], s.view(torch.uint8)[:, 0]) and torch.equal(codes.cpu()[0, 0, :3], c[:, 0])


@pytest.mark.parametrize("exp", [-64, -40, -12, -9, 0, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_finite_values_far_past_the_range_keep_their_sign(D, exp):
    """Every power of two that bf16 has, both signs, alone in its 16 values and with others: byte for byte the definition's."""
    powers = torch.arange(-126, 128).double().exp2()
    top = torch.tensor([torch.finfo(torch.bfloat16).max], dtype=torch.float64)
    peak = torch.cat([powers, top, -powers, -top])
    x = torch.zeros(peak.numel(), D // 16, 16, dtype=torch.float64)
    x[:, 0, 3] = peak                              # alone
    x[:, 1] = peak[:, None] * torch.tensor([1.0, -1.0, 0.5, -0.5, 0.25, -0.75, 0.0, 1.0] * 2, dtype=torch.float64)
    x[:, 2] = torch.randn(peak.numel(), 16, generator=gen(5), dtype=torch.float64)
    x[:, 2, 15] = -peak                            # beside small ones
    x = x.flatten(1).to(torch.bfloat16)[:, None]
    T, page = x.shape[0], 16
    N = -(-T // page)
    kc, vc, ks, vs = empty4(N, 1, page, D)
    less = 0.0 - x                                 # (zeros stay without a sign)
    dash.kv_write(x.to(DEV), less.to(DEV), kc, vc, torch.arange(T, device=DEV), k_scale=ks.view(E4M3), v_scale=vs.view(E4M3), k_exp=exp, v_exp=exp)
    no_error()
    for y, codes, scales in ((x, kc, ks), (less, vc, vs)):
        c, s = quantised4(y, exp)
        assert torch.equal(scales.cpu().flatten(0, 2)[:T], s.view(torch.uint8).flatten(0, 1))
        assert torch.equal(codes.cpu().flatten(0, 2)[:T], c.flatten(0, 1))


def zero_keys(c):
    c.k_cache.zero_()
    c.kw["k_exp"] = 64
    for k in c.k:
        k[:] = 0.0


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_large_queries_over_keys_of_zero_and_greatest_exponents(n, D):
    """Scores' scales far above the largest number: a score of zero stays zero, and every key weighs the same."""
    g = gen(14)
    c = paged4(g, [200, 77], 2, D, 16)
    zero_keys(c)
    q = randn(g, 2 * n, 8, D)
    q[:, 1::2] *= 2.0 ** 100
    q[n:, 3] = torch.finfo(torch.bfloat16).max
    o, lse = run_attn(c, q, [n, n])
    no_error()
    check_attn4(c, q, [n, n], o, lse)


@pytest.mark.parametrize("name", ["two_of_64", "two_of_128", "three_of_64", "three_of_128"])
def test_row_tiles_of_large_queries_over_keys_of_zero(name):
    c, q, n, window, causal = tile_inputs(name, seed=9)
    zero_keys(c)
    q[::2] *= 2.0 ** 100
    o, lse = run_attn(c, q, n, window=window, causal=causal)
    no_error()
    check_attn4(c, q, n, o, lse, window=window, causal=causal)
