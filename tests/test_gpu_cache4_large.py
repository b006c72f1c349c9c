"""Caches whose cells lie past 32-bit offsets, and the largest pools of rows."""
import random

import numpy as np
import pytest
import torch

from oracle import pages as PG
from tile_scheduling_persistent_gb300 import dash

from cache4_helpers import check_attn4, quantised4, values4
from serving_helpers import DEV, E4M3, Paged, no_error, randn, run_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 40])
def test_cells_past_4_gib(n):
    """Written, read, attended to and copied at the far end of a cache of more than 2^32 bytes."""
    Hq, Hkv, D, page, L = 8, 2, 128, 256, 700
    N = (1 << 32) // (Hkv * page * D // 2) + 8
    k, v = (torch.empty(N, Hkv, page, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty(N, Hkv, page, D // 16, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    kw = dict(k_scale=ks, v_scale=vs, k_exp=-2, v_exp=-1)
    g = torch.Generator().manual_seed(1)
    pages = [N - 1, N - 7, N - 3]
    x = randn(g, L, 2 * Hkv, D)
    j = torch.arange(L)
    slots = torch.tensor(pages)[j // page] * page + j % page
    d = x.to(DEV)
    dash.kv_write(d[:, :Hkv], d[:, Hkv:], k, v, slots.to(DEV), **kw)
    held = [values4(*quantised4(x[:, s], e), e).numpy() for s, e in ((slice(0, Hkv), -2), (slice(Hkv, None), -1))]
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    ko, vo = (torch.zeros(1, Hkv, L, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dash.kv_read(k, v, table, lens, ko, vo, **kw)
    for got, ref in ((ko, held[0]), (vo, held[1])):
        assert np.array_equal(got[0].transpose(0, 1).float().cpu().double().numpy(), ref)
    q = randn(g, n, Hq, D)
    c = Paged([held[0]], [held[1]], k, v, ks, vs, table, lens, kw)
    o, lse = run_attn(c, q, [n])
    check_attn4(c, q, [n], o, lse)
    dash.kv_copy([k], [v], torch.tensor([[p, i] for i, p in enumerate(pages)], dtype=torch.int32, device=DEV), k_scales=[ks], v_scales=[vs])
    near = Paged([held[0]], [held[1]], k, v, ks, vs, torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), lens, kw)
    o2, lse2 = run_attn(near, q, [n])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    no_error()


def test_the_most_rows_and_a_large_pool():
    rng = random.Random(2)
    R, page, width, N = 4096, 16, 40, 1 << 18
    order = rng.sample(range(N), R * 6)
    lens = [rng.randint(0, 16 * 5) for _ in range(R)]
    rows = [[order.pop() for _ in range(PG.pages_of(n, page))] for n in lens]
    refs = [0] * N
    for row in rows:
        for p in row:
            refs[p] += 1
    t = torch.full((R, width), -1, dtype=torch.int32)
    for r, row in enumerate(rows):
        t[r, :len(row)] = torch.tensor(row, dtype=torch.int32)
    t, l, c = t.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(refs, dtype=torch.int32, device=DEV)
    parents = [rng.randrange(R) for _ in range(R)]
    t1, l1 = torch.zeros_like(t), torch.zeros_like(l)
    dash.pages_fork(t, l, torch.tensor(parents, dtype=torch.int32, device=DEV), t1, l1, c, page)
    rows, lens, refs = PG.fork(rows, lens, parents, refs)
    new = [rng.choice([0, 1, 2, 200]) for _ in range(R)]
    T = sum(new)
    slots, pos = torch.zeros(T, dtype=torch.int64, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    copies, counts = torch.zeros(R, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    dash.pages_extend(t1, l1, c, page, slots, pos, copies, counts, cu_new=cu)
    rows, lens, refs, want, taken, at, where = PG.extend(rows, lens, refs, new, page)
    assert counts.tolist() == [len(want), taken] and copies[:len(want)].tolist() == [list(p) for p in want]
    assert slots.tolist() == where and pos.tolist() == at and l1.tolist() == lens and c.tolist() == refs
    got = t1.cpu().tolist()
    assert all(got[r][:len(row)] == row for r, row in enumerate(rows))
    moved, mc = torch.zeros(N // 2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    dash.pages_compact(t1, l1, c, page, moved, mc)
    rows, refs, moves, live = PG.compact(rows, refs)
    assert mc.tolist() == [len(moves), live] and c.tolist() == refs
    got = t1.cpu().tolist()
    assert all(got[r][:len(row)] == row for r, row in enumerate(rows))
    no_error()
