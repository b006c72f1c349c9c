"""Attention over the paged cache on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from tile_scheduling_persistent_gb300 import dash

from serving_helpers import DEV, check_attn, no_error, paged, randn, run_attn, same

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


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
    "chunk_many": (8, 8, 128, 64, [211 * i % 700 + 300 for i in range(30)], [17 * i % 300 + 17 for i in range(30)], None, 3),
    "group_128": (128, 1, 64, 16, [90, 300], [1, 3], None, 0),
}


def inputs(name, quant, seed=1):
    Hq, Hkv, D, page, lens, n, window, pad = CASES[name]
    g = gen(seed)
    c = paged(g, lens, Hkv, D, page, quant)
    return c, randn(g, sum(n) + pad, Hq, D), n, window


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("quant", [False, True])
def test_against_the_oracle(name, quant):
    c, q, n, window = inputs(name, quant)
    o, lse = run_attn(c, q, n, window=window)
    no_error()
    check_attn(c, q, n, o, lse, window=window)


@pytest.mark.parametrize("name", ["decode_ragged", "verify", "chunk_ragged", "mixed"])
@pytest.mark.parametrize("quant", [False, True])
def test_full_mask(name, quant):
    c, q, n, _ = inputs(name, quant, seed=2)
    o, lse = run_attn(c, q, n, causal=False)
    no_error()
    check_attn(c, q, n, o, lse, causal=False)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [False, True])
def test_every_page_size(page, D, quant):
    g = gen(3)
    c = paged(g, [page * 2 + 3, 300, 1], 2, D, page, quant)
    for n in ([1, 1, 1], [40, 33, 1]):
        q = randn(g, sum(n), 8, D)
        o, lse = run_attn(c, q, n)
        no_error()
        check_attn(c, q, n, o, lse)


@pytest.mark.parametrize("n", [[1, 1], [30, 90]])
@pytest.mark.parametrize("quant", [False, True])
def test_large_scores(n, quant):
    # scores of +-60 and more: the running maximum rises again and again, and most weights vanish.  A score's fp32
    # error grows with the absolute sum behind it; queries in few bits and keys of +-1 keep it exact.
    g = gen(4)
    D, Hkv = 128, 2
    c = paged(g, [700, 300], Hkv, D, 16, False)
    if quant:
        c = paged(g, [700, 300], Hkv, D, 16, True)
    q = (torch.randint(-6, 7, (sum(n), 8, D), generator=g).float()).to(torch.bfloat16)
    o, lse = run_attn(c, q, n)
    no_error()
    # |score error| <= 130 * 2^-23 * sum|q k| / sqrt(D) <= 130 * 2^-23 * 128 * 4 * 3.3 / 11.3 = 2.3e-3: the bound's fp32 part
    # (2^-10 A = 4 * 2^-12 A) becomes 2 * 2.3e-3 A; the rest is as in check_attn
    from oracle import serving as V
    at = 0
    for b, m in enumerate(n):
        ln = c.k[b].shape[0]
        ro, rl = V.attend(q[at:at + m].double().numpy(), c.k[b], c.v[b], ln - m)
        A, _ = V.attend(q[at:at + m].double().numpy(), c.k[b], np.abs(c.v[b]), ln - m)
        d = np.abs(o[at:at + m].float().cpu().double().numpy() - ro)
        assert (d <= (2.0 ** -8 + 5e-3) * A + 2.0 ** -8 * np.abs(ro)).all()
        assert np.abs(lse[at:at + m].cpu().double().numpy() - rl).max() <= 2.5e-3
        at += m


@pytest.mark.parametrize("name", ["decode_ragged", "verify", "chunk_ragged", "mixed"])
def test_strided_queries_no_lse_given_workspace(name):
    Hq, Hkv, D, page, lens, n, window, pad = CASES[name]
    c, q, n, window = inputs(name, False, seed=5)
    ref, _ = run_attn(c, q, n, window=window)
    T = q.shape[0]
    rows = torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)   # a projection's rows
    rows[:, :Hq] = q.to(DEV)
    heads = q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)             # heads before tokens
    need = dash.attn_paged_workspace(len(n), T, Hq, Hkv, D, max(n), c.table.shape[1] * page)
    for x in (rows[:, :Hq], heads):
        o = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device=DEV)
        dash.attn_paged(x, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=max(n), workspace=ws)
        no_error()
        assert same(o, ref)


def test_equal_counts_need_no_cu():
    g = gen(6)
    c = paged(g, [100, 7, 64], 2, 128, 16, True)
    for n in (1, 3, 20):
        q = randn(g, 3 * n, 8, 128)
        a = run_attn(c, q, [n] * 3)
        b = run_attn(c, q, [n] * 3, use_cu=False, max_q=None)
        d = torch.full_like(a[0], 77.0)
        dash.attn_paged(q.to(DEV), c.k_cache, c.v_cache, c.table, c.lens, d, **c.kw)
        assert same(a[0], b[0]) and same(a[1], b[1]) and same(a[0], d)
        check_attn(c, q, [n] * 3, *a)


@pytest.mark.parametrize("quant", [False, True])
def test_a_sequence_does_not_depend_on_its_batch(quant):
    # alone, in a batch, in another order, with a larger max_q and a wider table: the same bits
    Hq, Hkv, D, page = 16, 4, 128, 16
    g = gen(7)
    lens, n = [2600, 40, 900, 1500], [1, 1, 3, 200]
    c = paged(g, lens, Hkv, D, page, quant, max_len=4000)
    q = randn(g, sum(n), Hq, D)
    first = [0, 1, 2, 5]
    o, lse = run_attn(c, q, n)
    no_error()
    again = run_attn(c, q, n)
    assert same(o, again[0]) and same(lse, again[1])

    def part(order, width, max_q):
        sub = [q[first[b]:first[b] + n[b]] for b in order]
        m = [n[b] for b in order]
        import copy
        d = copy.copy(c)
        d.table, d.lens = c.table[order, :width].contiguous(), c.lens[order].contiguous()
        oo, ll = run_attn(d, torch.cat(sub), m, max_q=max_q)
        no_error()
        at = 0
        for b in order:
            assert same(oo[at:at + n[b]], o[first[b]:first[b] + n[b]]) and same(ll[at:at + n[b]], lse[first[b]:first[b] + n[b]]), (order, b)
            at += n[b]

    full = c.table.shape[1]
    for b in range(4):
        part([b], -(-lens[b] // page), n[b])
        part([b], full, 300)
    part([3, 1, 0, 2], full, 200)
    part([0, 1], 2600 // page + 1, 1)


def test_stale_and_freed_pages_do_not_matter():
    # pages wholly before the window are freed (table entry -1), their cells and those past the length hold NaN or infinities
    g = gen(8)
    for quant in (False, True):
        for n in ([1, 1], [60, 25]):
            c = paged(g, [1000, 611], 2, 128, 16, quant)
            window = 200
            q = randn(g, sum(n), 8, 128)
            table = c.table.clone()
            for b, ln in enumerate([1000, 611]):
                gone = max(0, ln - n[b] + 1 - window) // 16
                for p in table[b, :gone].tolist():
                    if quant:
                        c.v_cache.view(torch.uint8)[p] = 0x7f
                        c.v_scale[p] = float("inf")
                    else:
                        c.v_cache[p] = float("inf")
                        c.k_cache[p] = float("nan")
                table[b, :gone] = -1
            c.table = table
            o, lse = run_attn(c, q, n, window=window)
            no_error()
            check_attn(c, q, n, o, lse, window=window)


@pytest.mark.parametrize("n", [[1, 1, 1], [40, 1, 60]])
@pytest.mark.parametrize("quant", [False, True])
def test_bad_pages_and_lengths_are_reported_and_stay_in_their_sequence(n, quant):
    g = gen(9)
    c = paged(g, [300, 200, 400], 2, 128, 16, quant)
    q = randn(g, sum(n), 8, 128)
    o, lse = run_attn(c, q, n)
    no_error()
    good = c.table.clone()
    for bad in (10 ** 6, c.k_cache.shape[0], -1, -2 ** 31):
        c.table = good.clone()
        c.table[1, 3] = bad
        o2, lse2 = run_attn(c, q, n)
        code, info = dash.get_status_paged()
        assert code == dash.ERR_PAGE and info[:2] == [3, 1] and info[2] == bad and info[3] == c.k_cache.shape[0]
        no_error()
        for a, b in ((0, n[0]), (n[0] + n[1], sum(n))):
            assert same(o[a:b], o2[a:b]) and same(lse[a:b], lse2[a:b])
    c.table = good
    lens = c.lens.clone()
    for ln in (good.shape[1] * 16 + 1, 2 ** 31 - 1, -1):
        c.lens = lens.clone()
        c.lens[1] = ln
        c.table = good.clone()
        c.table[1][c.table[1] < 0] = 0                    # the length alone is wrong
        o2, lse2 = run_attn(c, q, n)
        code, info = dash.get_status_paged()
        assert code == dash.ERR_PAGE and info[:2] == [3, 1] and info[2] == ln
        for a, b in ((0, n[0]), (n[0] + n[1], sum(n))):
            assert same(o[a:b], o2[a:b]) and same(lse[a:b], lse2[a:b])


@pytest.mark.parametrize("n,max_q", [([2, 1], 1), ([30, 1], 4), ([90, 40], 89)])
def test_more_new_tokens_than_said_are_reported(n, max_q):
    g = gen(10)
    c = paged(g, [100, 120], 2, 64, 16, False)
    q = randn(g, sum(n), 4, 64)
    o, _ = run_attn(c, q, n)
    no_error()
    o2, _ = run_attn(c, q, n, max_q=max_q)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info == [3, 0, n[0], max_q]
    assert same(o[n[0]:], o2[n[0]:])


def test_rows_past_the_buffers_are_reported():
    # cu_q runs past T: what does not exist is neither read nor written
    g = gen(11)
    c = paged(g, [100, 120], 2, 64, 16, False)
    for n in ([1, 1], [3, 60]):
        q = randn(g, sum(n) + 40, 4, 64)
        o, lse = run_attn(c, q[:sum(n)], n)
        T = n[0]
        big = torch.full((sum(n) + 40, 4, 64), 77.0, dtype=torch.bfloat16, device=DEV)
        cu = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV)
        dash.attn_paged(q.to(DEV)[:T], c.k_cache, c.v_cache, c.table, c.lens, big[:T], cu_q=cu, max_q=max(n))
        code, info = dash.get_status_paged()
        assert code == dash.ERR_PAGE and info[:2] == [3, 1]
        assert same(big[:T], o[:T]) and (big[T:] == 77.0).all()


@pytest.mark.parametrize("name", ["decode_ragged", "mixed"])
def test_captured_and_replayed_with_new_lengths(name):
    Hq, Hkv, D, page, lens, n, window, pad = CASES[name]
    c, q, n, window = inputs(name, True, seed=12)
    qd, o = q.to(DEV), torch.full(q.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 77.0, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    call = lambda: dash.attn_paged(qd, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=max(n), lse=lse, **c.kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shorter in (0, 1):
        now = [max(ln - 30 * shorter, min(ln, m)) for ln, m in zip(lens, n)]
        c.lens.copy_(torch.tensor(now, dtype=torch.int32))
        d = type(c)([k[:m] for k, m in zip(c.k, now)], [v[:m] for v, m in zip(c.v, now)], c.k_cache, c.v_cache, c.k_scale,
                    c.v_scale, c.table, c.lens, c.kw)
        o.fill_(77.0)
        lse.fill_(77.0)
        graph.replay()
        no_error()
        check_attn(d, q, n, o, lse)


def test_two_streams_at_once():
    g = gen(13)
    c = paged(g, [3000, 2000, 100], 4, 128, 16, True)
    work = []
    for n in ([1, 1, 1], [100, 1, 30]):
        q = randn(g, sum(n), 16, 128).to(DEV)
        work.append((q, n, run_attn(c, q, n)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(12):
        q, n, _ = work[i % 2]
        s = streams[i % 4]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        o = torch.empty_like(q)
        s.wait_stream(torch.cuda.current_stream())
        dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=max(n), stream=s, **c.kw)
        got.append((o, work[i % 2][2][0], cu))
    torch.cuda.synchronize()
    no_error()
    for o, ref, _ in got:
        assert same(o, ref)


def test_cache_beyond_32_bit_offsets():
    # 2.2e9 elements in each of k and v: cells at the far end
    page, Hkv, D = 128, 8, 128
    N = 2 ** 31 // (page * Hkv * D) + 1200
    g = gen(14)
    c = paged(g, [300, 260], Hkv, D, page, False)
    k, v = (torch.empty(N, Hkv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    used = c.table >= 0
    far = torch.where(used, N - 1 - c.table, c.table)
    idx = c.table[used].long()
    k[N - 1 - idx] = c.k_cache[idx]
    v[N - 1 - idx] = c.v_cache[idx]
    for n in ([1, 1], [40, 50]):
        q = randn(g, sum(n), 16, D)
        ref = run_attn(c, q, n)
        o = torch.empty_like(ref[0])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        dash.attn_paged(q.to(DEV), k, v, far.contiguous(), c.lens, o, cu_q=cu, max_q=max(n))
        no_error()
        assert same(o, ref[0])


def test_binding_refuses():
    g = gen(15)
    c = paged(g, [30, 40], 2, 64, 16, False)
    e = paged(g, [30, 40], 2, 64, 16, True)
    q = randn(g, 2, 4, 64).to(DEV)
    base = dict(q=q, k_cache=c.k_cache, v_cache=c.v_cache, block_table=c.table, kv_lens=c.lens, o=torch.empty_like(q))
    bad = [dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q[:, :, :32]), dict(o=torch.empty_like(q)[:1]), dict(kv_lens=c.lens.long()),
           dict(block_table=c.table[:1]), dict(block_table=c.table.long()), dict(k_scale=e.k_scale), dict(k_cache=e.k_cache),
           dict(k_cache=e.k_cache, v_cache=e.v_cache), dict(k_cache=e.k_cache, v_cache=e.v_cache, k_scale=e.k_scale, v_scale=e.v_scale[:1]),
           dict(v_cache=c.v_cache[:1]), dict(cu_q=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(lse=torch.empty(2, 3, device=DEV)),
           dict(window=0), dict(window=3, causal=False), dict(q=q[:, :3], o=torch.empty_like(q[:, :3])), dict(max_q=0),
           dict(q=q.cpu()), dict(kv_lens=c.lens.cpu())]
    for kw in bad:
        with pytest.raises(dash.DashError):
            dash.attn_paged(**{**base, **kw})
    dash.attn_paged(**base)
    no_error()
    # nothing to do: no tokens, no sequences
    dash.attn_paged(**{**base, **dict(q=q[:0], o=torch.empty_like(q[:0]), cu_q=torch.zeros(3, dtype=torch.int32, device=DEV))})
    dash.attn_paged(**{**base, **dict(q=q[:0], o=torch.empty_like(q[:0]), kv_lens=c.lens[:0], block_table=c.table[:0])})
    no_error()
