"""The pages of a cache on the GPU -- forked, extended, dropped, moved and copied -- against plain Python."""
import random

import pytest
import torch

from oracle import pages as PG
from tile_scheduling_persistent_gb300 import dash

from cache4_helpers import paged4
from serving_helpers import DEV, E4M3, no_error, paged

pytestmark = pytest.mark.gpu

MARK = -5   # what entries and lists hold where nothing is written


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


class Pool:
    """The state on the GPU and in plain Python."""

    def __init__(self, rng, pages, page, width, rows, most):
        self.page, self.width, self.N = page, width, pages
        order = list(range(pages))
        rng.shuffle(order)
        self.lens = [rng.choice([0, page, rng.randint(0, most)]) for _ in range(rows)]
        self.rows = [[order.pop() for _ in range(PG.pages_of(n, page))] for n in self.lens]
        self.refs = [0] * pages
        for row in self.rows:
            for p in row:
                self.refs[p] += 1
        self.up()

    def up(self):
        self.t = torch.full((len(self.rows), self.width), MARK, dtype=torch.int32)
        for r, row in enumerate(self.rows):
            self.t[r, :len(row)] = torch.tensor(row, dtype=torch.int32)
        self.t = self.t.to(DEV)
        self.l, self.c = ints(self.lens), ints(self.refs)

    def check(self, behind=None):
        """behind: what the entries behind a row's pages hold (None: anything)."""
        t, lens = self.t.cpu().tolist(), self.l.cpu().tolist()
        assert lens == self.lens and self.c.cpu().tolist() == self.refs
        for r, row in enumerate(self.rows):
            assert t[r][:len(row)] == row, r
            assert behind is None or t[r][len(row):] == [behind] * (self.width - len(row))

    def fork(self, parents):
        out = torch.full((len(parents), self.width), MARK, dtype=torch.int32, device=DEV)
        lens = torch.full((len(parents),), MARK, dtype=torch.int32, device=DEV)
        dash.pages_fork(self.t, self.l, ints(parents), out, lens, self.c, self.page)
        self.rows, self.lens, self.refs = PG.fork(self.rows, self.lens, parents, self.refs)
        self.t, self.l = out, lens
        self.check(-1)

    def extend(self, n_new, pad=0, even=False):
        R, T = len(n_new), sum(n_new) + pad
        slots, pos = torch.full((T,), 7, dtype=torch.int64, device=DEV), torch.full((T,), 7, dtype=torch.int32, device=DEV)
        copies, counts = torch.full((R, 2), MARK, dtype=torch.int32, device=DEV), ints([MARK, MARK])
        cu = None if even else ints([sum(n_new[:i]) for i in range(R + 1)])
        dash.pages_extend(self.t, self.l, self.c, self.page, slots, pos, copies, counts, cu_new=cu)
        got = PG.extend(self.rows, self.lens, self.refs, n_new, self.page)
        if got is None:
            assert counts.tolist() == [0, 0] and slots.tolist() == [-1] * T and copies.flatten().tolist() == [MARK] * (2 * R)
            code, info = dash.get_status_paged()
            assert code == dash.ERR_NOMEM and info[0] == 5 and info[2] > info[3] == self.refs.count(0)
        else:
            self.rows, self.lens, self.refs, want, taken, at, where = got
            assert counts.tolist() == [len(want), taken]
            assert copies.tolist() == [list(p) for p in want] + [[MARK, MARK]] * (R - len(want))
            assert slots.tolist() == where + [-1] * pad and pos.tolist() == at + [0] * pad
        self.check()
        return slots, copies, counts

    def compact(self, in_place):
        copies, counts = torch.full((self.N // 2, 2), MARK, dtype=torch.int32, device=DEV), ints([MARK, MARK])
        t, c = (None, None) if in_place else (torch.full_like(self.t, 99), torch.full_like(self.c, 99))
        dash.pages_compact(self.t, self.l, self.c, self.page, copies, counts, table_out=t, refs_out=c)
        self.rows, self.refs, moves, L = PG.compact(self.rows, self.refs)
        assert counts.tolist() == [len(moves), L]
        assert copies.tolist() == [list(m) for m in moves] + [[MARK, MARK]] * (self.N // 2 - len(moves))
        if not in_place:
            self.t, self.c = t, c
        self.check()
        return copies, counts


@pytest.mark.parametrize("rows,pages,page", [(1, 9, 16), (5, 60, 32), (40, 700, 16), (130, 9000, 64), (1100, 5000, 16), (3, 40003, 256)])
def test_random_steps(rows, pages, page):
    rng = random.Random(rows)
    width = max(4, pages // max(rows, 4))
    p = Pool(rng, pages, page, width, rows, min(page * width // 2, page * (pages // (2 * rows) + 1) - 1, 4000))
    for step in range(8):
        n = len(p.rows)
        kind = step % 4
        if kind == 0:      # some dropped, some forked
            want = rng.randint(1, rows + 2)
            p.fork([rng.choice([-1, rng.randrange(n), rng.randrange(n), min(i, n - 1)]) for i in range(want)])
        elif kind == 3:
            p.compact(step == 3)
        else:
            most = rng.choice([1, 3, page + 2])
            new = [min(rng.choice([0, 1, rng.randint(0, most)]), width * page - x) for x in p.lens]
            p.extend(new, pad=rng.choice([0, 3]))
    no_error()


def test_every_row_goes_on_in_one_shared_page():
    """The first keeps it where nobody else holds it, and not where a kept prefix does."""
    for kept in (0, 1):
        p = Pool(random.Random(0), 30, 16, 4, 1, 0)
        p.rows, p.lens = [[7, 3]], [21]
        p.refs = [0] * 30
        p.refs[7], p.refs[3] = 1 + kept, 1 + kept
        p.up()
        p.fork([0, 0, -1, 0])
        _, copies, counts = p.extend([1, 12, 0, 2])
        assert counts[0] == 2 + kept and p.refs[3] == 1 + (kept and 0)
        no_error()


def test_the_same_new_tokens_for_every_row_and_no_rows():
    p = Pool(random.Random(3), 50, 16, 8, 6, 60)
    p.extend([5] * 6, even=True)
    dash.pages_extend(p.t[:0], p.l[:0], p.c, 16, ints([], torch.int64), ints([]), ints([]).view(0, 2), torch.zeros(2, dtype=torch.int32, device=DEV))
    dash.pages_fork(p.t[:0], p.l[:0], ints([]), torch.empty(0, 8, dtype=torch.int32, device=DEV), ints([]), p.c, 16)
    p.check()
    no_error()


def test_too_few_pages_change_nothing():
    p = Pool(random.Random(4), 12, 16, 8, 3, 40)
    p.extend([120 - n for n in p.lens])
    p.extend([1, 0, 0])
    no_error()


def test_rows_out_of_range_are_reported_and_left():
    p = Pool(random.Random(5), 40, 16, 4, 4, 0)
    p.rows, p.lens = [[1], [2], [3, 4], [5, 6, 7, 8]], [3, 9, 20, 60]
    p.refs = [0] * 40
    for row in p.rows:
        for q in row:
            p.refs[q] = 1
    p.up()
    slots, pos, copies, counts = ints([9] * 12, torch.int64), ints([9] * 12), ints([[MARK] * 2] * 4), ints([9, 9])
    p.l[1] = -4                                          # a length below zero; the last row's pages would pass the table
    dash.pages_extend(p.t, p.l, p.c, 16, slots, pos, copies, counts, cu_new=ints([0, 2, 4, 6, 12]))
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info in ([5, 1, -4, 64], [5, 3, 66, 64])
    assert slots.tolist() == [16 + 3, 16 + 4, -1, -1, 64 + 4, 64 + 5] + [-1] * 6 and counts.tolist() == [0, 0]
    assert p.l.tolist() == [5, -4, 22, 60] and p.c.tolist() == p.refs
    p.l[1] = 9
    p.t[0, 0] = 40                                       # a last page out of range
    dash.pages_extend(p.t, p.l, p.c, 16, slots, pos, copies, counts, cu_new=ints([0, 2, 4, 6, 6]))
    assert dash.get_status_paged() == (dash.ERR_PAGE, [5, 0, 40, 40])
    assert slots.tolist() == [-1, -1, 41, 42, 64 + 6, 64 + 7] + [-1] * 6 and p.l.tolist() == [5, 11, 24, 60]
    dash.pages_extend(p.t, p.l, p.c, 16, slots, pos, copies, counts, cu_new=ints([0, 2, 1, 13, 13]))   # counts that decrease, or pass T
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info[0] == 5
    assert p.l.tolist() == [5, 11, 24, 60] and slots.tolist()[2:] == [-1] * 10
    no_error()


def test_fork_reports_what_is_out_of_range():
    p = Pool(random.Random(6), 20, 16, 4, 3, 40)
    p.rows, p.lens, p.refs = [[1, 2], [3], [4]], [20, 16, 5], [0, 1, 1, 1, 1] + [0] * 15
    p.up()
    out, lens = torch.full((2, 4), 9, dtype=torch.int32, device=DEV), ints([9, 9])
    dash.pages_fork(p.t, p.l, ints([3, 0]), out, lens, p.c, 16)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 0, 3, 3])
    assert out.tolist() == [[-1] * 4, [1, 2, -1, -1]] and lens.tolist() == [0, 20] and p.c.tolist() == [0, 1, 1, 0, 0] + [0] * 15
    p.up()
    p.t[0, 1] = 20
    dash.pages_fork(p.t, p.l, ints([1]), out[:1], lens[:1], p.c, 16)      # rows 0 and 2 are dropped
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 0, 20, 20])
    assert p.c.tolist() == [0, 0, 1, 1, 0] + [0] * 15
    dash.pages_fork(p.t[2:].clone(), ints([5]), ints([-1]), out[:1], lens[:1], p.c, 16)   # its page is free already
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 0, 0, -1])
    p.up()
    p.l[1] = 65
    dash.pages_fork(p.t, p.l, ints([0, 2]), out, lens, p.c, 16)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 1, 65, 64])
    assert p.c.tolist() == p.refs
    no_error()


def test_compact_reports_an_entry_of_a_free_page():
    p = Pool(random.Random(7), 20, 16, 4, 2, 0)
    p.rows, p.lens, p.refs = [[18], [11]], [16, 3], [0] * 20
    p.refs[18] = 1                                       # page 11 is free
    p.up()
    copies, counts = ints([[MARK] * 2] * 10), ints([9, 9])
    dash.pages_compact(p.t, p.l, p.c, 16, copies, counts)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [6, 1, 11, 20])
    assert counts.tolist() == [1, 1] and copies.tolist()[0] == [18, 0] and p.t[:, 0].tolist() == [0, 11] and p.c.tolist() == [1] + [0] * 19
    no_error()


@pytest.mark.parametrize("N", [1, 2, 3, 4096, 4097, 100001])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_compact_pools(N, share):
    g = torch.Generator().manual_seed(N)
    refs = (torch.rand(N, generator=g) < share).to(torch.int32) * torch.randint(1, 9, (N,), generator=g, dtype=torch.int32)
    live = torch.nonzero(refs)[:, 0]
    table = live[torch.randperm(live.numel(), generator=g)].to(torch.int32)
    lens = [16 * table.numel()]
    t = torch.cat([table, torch.tensor([MARK], dtype=torch.int32)])[None].to(DEV)
    copies, counts = torch.full((N // 2, 2), MARK, dtype=torch.int32, device=DEV), ints([9, 9])
    out, ref_out = torch.empty_like(t), torch.empty(N, dtype=torch.int32, device=DEV)
    dash.pages_compact(t, ints(lens), refs.to(DEV), 16, copies, counts, table_out=out, refs_out=ref_out)
    rows, want, moves, L = PG.compact([table.tolist()], refs.tolist())
    assert counts.tolist() == [len(moves), L] and copies[:len(moves)].tolist() == [list(m) for m in moves]
    assert (copies[len(moves):] == MARK).all() and ref_out.tolist() == want and out[0].tolist() == rows[0] + [MARK]
    no_error()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("D,Hkv,page,layers", [(64, 1, 16, 1), (128, 3, 32, 3), (64, 2, 256, 2), (128, 8, 64, 70)])
def test_copy(kind, D, Hkv, page, layers):
    N = 9
    g = torch.Generator().manual_seed(1)
    bits = lambda *shape: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).to(DEV)  # noqa: E731
    width = {"bf16": 2 * D, "e4m3": D, "e2m1": D // 2}[kind]
    view = {"bf16": torch.bfloat16, "e4m3": E4M3, "e2m1": torch.uint8}[kind]
    cells = [[bits(N, Hkv, page, width) for _ in range(layers)] for _ in range(2)]
    scales = [[bits(N, Hkv, page, 4 if kind == "e4m3" else D // 16) for _ in range(layers)] for _ in range(2)] if kind != "bf16" else [[], []]
    every = cells[0] + cells[1] + scales[0] + scales[1]
    before = [t.clone() for t in every]
    pairs = ints([[3, 0], [3, 8], [5, 2], [7, 6]])
    as_scales = [[s.view(torch.float32).squeeze(-1) if kind == "e4m3" else s.view(E4M3) for s in x] for x in scales]
    call = lambda pairs, counts: dash.kv_copy(*[[t.view(view) for t in x] for x in cells], pairs, counts,  # noqa: E731
                                              k_scales=as_scales[0], v_scales=as_scales[1])
    call(pairs, ints([3, 99]))
    for a, b in zip(every, before):
        b[0], b[8], b[2] = b[3].clone(), b[3].clone(), b[5].clone()
        assert torch.equal(a, b)
    call(pairs, None)
    call(pairs, ints([99, 0]))
    for a, b in zip(every, before):
        b[6] = b[7].clone()
        assert torch.equal(a, b)
    call(pairs[:0], None)
    no_error()
    call(ints([[0, 9], [-1, 2], [4, 1]]), None)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info in ([7, 0, 9, 9], [7, 1, -1, 9])
    for a, b in zip(every, before):
        b[1] = b[4].clone()
        assert torch.equal(a, b)


@pytest.mark.parametrize("make", [lambda g: paged(g, [150, 37, 0, 64], 2, 64, 16, False, extra_pages=60),
                                  lambda g: paged4(g, [150, 37, 0, 64], 2, 128, 32, extra_pages=60)], ids=["bf16", "e2m1"])
def test_in_a_captured_graph_and_on_another_stream(make):
    """Fork, extend, copy and drop, captured: every replay leaves what the calls leave, from the state that it finds."""
    c = make(torch.Generator().manual_seed(2))
    page, N = c.k_cache.shape[2], c.k_cache.shape[0]
    held = torch.arange(c.table.shape[1]) < (c.lens.cpu()[:, None] + page - 1) // page
    refs = torch.zeros(N, dtype=torch.int32)
    refs[c.table.cpu()[held].long()] = 1
    table = torch.cat([c.table, torch.full((4, 4), -1, dtype=torch.int32, device=DEV)], 1)
    c4 = dict(k_scales=[c.k_scale], v_scales=[c.v_scale]) if c.k_scale is not None else {}
    parents, kept = ints([0, 1, 2, 3, 0, 0, 1, 3]), ints([0, 1, 2, 3] + [-1] * 4)
    cu = ints([0, 0, 0, 0, 0, 5, 21, 22, 40])
    s = dict(t1=torch.zeros(8, table.shape[1], dtype=torch.int32, device=DEV), l1=ints([0] * 8), t2=torch.zeros(8, table.shape[1], dtype=torch.int32, device=DEV),
             l2=ints([0] * 8), slots=torch.zeros(40, dtype=torch.int64, device=DEV), pos=ints([0] * 40), copies=ints([[0, 0]] * 8), counts=ints([0, 0]),
             refs=refs.to(DEV))

    def step():
        dash.pages_fork(table, c.lens, parents, s["t1"], s["l1"], s["refs"], page)
        dash.pages_extend(s["t1"], s["l1"], s["refs"], page, s["slots"], s["pos"], s["copies"], s["counts"], cu_new=cu)
        dash.kv_copy([c.k_cache], [c.v_cache], s["copies"], s["counts"], **c4)
        dash.pages_fork(s["t1"], s["l1"], kept, s["t2"], s["l2"], s["refs"], page)

    step()
    want = {n: t.clone() for n, t in s.items()}
    cells = [t.view(torch.uint8).clone() for t in (c.k_cache, c.v_cache)]   # (as bytes: cells without a token are NaN)
    assert want["counts"][0] > 0 and torch.equal(want["refs"].cpu(), refs)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in s.values():
        if t is not s["refs"]:
            t.fill_(55)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for n, t in s.items():
        done = slice(int(want["counts"][0])) if n == "copies" else slice(None)
        assert torch.equal(t[done], want[n][done]), n
    assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip((c.k_cache, c.v_cache), cells))
    no_error()


def test_a_last_page_that_counts_as_free_is_reported():
    p = Pool(random.Random(8), 20, 16, 4, 2, 0)
    p.rows, p.lens, p.refs = [[4], [9]], [3, 5], [0] * 20
    p.refs[9] = 1                                        # page 4 is free
    p.up()
    slots, pos, copies, counts = ints([9] * 2, torch.int64), ints([9] * 2), ints([[MARK] * 2] * 2), ints([9, 9])
    dash.pages_extend(p.t, p.l, p.c, 16, slots, pos, copies, counts)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [5, 0, 0, 1])
    assert slots.tolist() == [-1, 149] and p.l.tolist() == [3, 6] and counts.tolist() == [0, 0]
    no_error()


def test_copy_of_layers_in_one_tensor():
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randint(0, 256, (3, 5, 2, 16, 32), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
    ks, vs = (torch.randint(0, 256, (3, 5, 2, 16, 4), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
    want = [t.clone() for t in (k, v, ks, vs)]
    for t in want:
        t[:, 1] = t[:, 4].clone()
    dash.kv_copy(k, v, ints([[4, 1]]), k_scales=ks.view(E4M3), v_scales=vs.view(E4M3))
    assert all(torch.equal(a, b) for a, b in zip((k, v, ks, vs), want))
    no_error()


def test_calls_on_two_streams_at_once():
    """Pools of their own on streams of their own, without waiting for one another."""
    pools = [Pool(random.Random(s), 600, 16, 20, 30, 100) for s in (21, 22)]
    streams = [torch.cuda.Stream() for _ in pools]
    torch.cuda.synchronize()
    work = []
    for p, st in zip(pools, streams):
        R = len(p.rows)
        a = dict(par=ints(list(range(R)) + [0, 0, 3]), t1=torch.zeros(R + 3, 20, dtype=torch.int32, device=DEV), l1=ints([0] * (R + 3)),
                 slots=torch.zeros(2 * (R + 3), dtype=torch.int64, device=DEV), pos=ints([0] * (2 * (R + 3))), copies=ints([[MARK] * 2] * (R + 3)),
                 counts=ints([0, 0]), moved=ints([[MARK] * 2] * 300), mc=ints([0, 0]))
        work.append(a)
    torch.cuda.synchronize()
    for p, st, a in zip(pools, streams, work):
        with torch.cuda.stream(st):
            dash.pages_fork(p.t, p.l, a["par"], a["t1"], a["l1"], p.c, 16)
            dash.pages_extend(a["t1"], a["l1"], p.c, 16, a["slots"], a["pos"], a["copies"], a["counts"])
            dash.pages_compact(a["t1"], a["l1"], p.c, 16, a["moved"], a["mc"])
    torch.cuda.synchronize()
    for p, a in zip(pools, work):
        rows, lens, refs = PG.fork(p.rows, p.lens, a["par"].tolist(), p.refs)
        rows, lens, refs, want, taken, at, where = PG.extend(rows, lens, refs, [2] * len(rows), 16)
        assert a["slots"].tolist() == where and a["counts"].tolist() == [len(want), taken]
        p.rows, p.refs, moves, live = PG.compact(rows, refs)
        p.lens, p.t, p.l = lens, a["t1"], a["l1"]
        assert a["mc"].tolist() == [len(moves), live]
        p.check()
    no_error()


def test_fork_reports_a_length_out_of_range_of_a_row_that_goes_on():
    p = Pool(random.Random(6), 20, 16, 4, 3, 40)
    p.rows, p.lens, p.refs = [[1, 2], [3], [4]], [20, 16, 5], [0, 1, 1, 1, 1] + [0] * 15
    p.up()
    p.l[1] = -1
    out, lens = torch.full((3, 4), 9, dtype=torch.int32, device=DEV), ints([9, 9, 9])
    dash.pages_fork(p.t, p.l, ints([0, 1, 2]), out, lens, p.c, 16)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 1, -1, 64])
    assert out.tolist() == [[1, 2, -1, -1], [-1] * 4, [4, -1, -1, -1]] and lens.tolist() == [20, 0, 5] and p.c.tolist() == p.refs
    no_error()


def test_rows_that_overlap_may_need_more_pages_than_32_bits_count():
    """Every other row's tokens run backwards, which is reported; the others have 2^24 tokens each, 2^31 pages in all."""
    rows, T = 4096, 1 << 24
    cu = ints([0, T] * (rows // 2) + [0])
    lens, refs = ints([0] * rows), ints([0, 1] * 50)
    table = torch.empty((rows, T // 16), dtype=torch.int32, device=DEV)   # no entry is read
    slots, pos = torch.full((T,), 9, dtype=torch.int64, device=DEV), torch.full((T,), 9, dtype=torch.int32, device=DEV)
    copies, counts = torch.full((rows, 2), MARK, dtype=torch.int32, device=DEV), ints([9, 9])
    dash.pages_extend(table, lens, refs, 16, slots, pos, copies, counts, cu_new=cu)
    assert dash.get_status_paged()[0] in (dash.ERR_PAGE, dash.ERR_NOMEM)
    assert counts.tolist() == [0, 0] and (lens == 0).all() and refs.tolist() == [0, 1] * 50
    assert (slots == -1).all() and (copies == MARK).all()
    no_error()


@pytest.mark.parametrize("N", [30, 20000])
@pytest.mark.parametrize("refs", [1, 2])
def test_rows_that_go_on_in_a_page_of_fewer_holders_are_reported_and_left(refs, N):
    """refs + 1 rows go on in page 7; the row behind them takes the lowest free page, in every run."""
    p = Pool(random.Random(8), N, 16, 4, 1, 0)
    p.rows, p.lens = [[3], [9]] + [[7]] * (refs + 1) + [[5]], [5, 7] + [2, 9, 15][:refs + 1] + [16]
    p.refs = [0] * N
    p.refs[3], p.refs[9], p.refs[7], p.refs[5] = 1, 2, refs, 1
    p.up()
    R = len(p.rows)
    for _ in range(3):
        t, lens, c = p.t.clone(), p.l.clone(), p.c.clone()
        slots, pos, copies, counts = ints([9] * R, torch.int64), ints([9] * R), ints([[MARK] * 2] * R), ints([9, 9])
        dash.pages_extend(t, lens, c, 16, slots, pos, copies, counts)
        code, info = dash.get_status_paged()
        assert code == dash.ERR_PAGE and info[0] == 5 and 2 <= info[1] <= 2 + refs and info[2:] == [refs, refs + 1]
        no_error()
        assert slots.tolist() == [53, 7] + [-1] * (refs + 1) + [16] and pos.tolist() == [5, 7] + [0] * (refs + 1) + [16]
        assert lens.tolist() == [6, 8] + p.lens[2:2 + refs + 1] + [17]
        assert counts.tolist() == [1, 2] and copies.tolist() == [[9, 0]] + [[MARK] * 2] * (R - 1)
        want = list(p.refs)
        want[0], want[1], want[9] = 1, 1, 1
        assert c.tolist() == want
        rows = p.t.tolist()
        rows[1][0], rows[-1][1] = 0, 1
        assert t.tolist() == rows


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("N,at", [(20, 2), (9000, 4097), (40000, 9001), (40000, 12)])
def test_compact_reports_an_entry_of_a_free_page_below_the_pages_in_use(N, at, in_place):
    """The free page is where another row's page goes: the entry stays as it is, and is reported."""
    refs = [0] * N
    for q in range(at + 1):
        refs[q] = 1
    refs[at] = 0
    refs[N - 1] = refs[N - 2] = 1                        # at + 2 pages in use; page `at` and the one behind it are free
    rows = [[N - 1], [at], [0], [N - 2]]
    t, lens, c = ints([r + [MARK] for r in rows]), ints([16, 3, 16, 9]), ints(refs)
    copies, counts = torch.full((N // 2, 2), MARK, dtype=torch.int32, device=DEV), ints([9, 9])
    to, co = (None, None) if in_place else (torch.full_like(t, 99), torch.full_like(c, 99))
    dash.pages_compact(t, lens, c, 16, copies, counts, table_out=to, refs_out=co)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [6, 1, at, N])
    no_error()
    assert counts.tolist() == [2, at + 2] and copies[:2].tolist() == [[N - 2, at], [N - 1, at + 1]]
    assert (t if in_place else to).tolist() == [[at + 1, MARK], [at, MARK], [0, MARK], [at, MARK]]
    assert (c if in_place else co).tolist() == [1] * (at + 2) + [0] * (N - at - 2)


@pytest.mark.parametrize("entry", [20, -3])
@pytest.mark.parametrize("parents", [[0, 1, 2], [2, 1], [1, -1], [2, 0, 1, 1]])
def test_fork_reports_an_entry_out_of_range_of_a_row_that_goes_on(parents, entry):
    p = Pool(random.Random(6), 20, 16, 4, 3, 40)
    p.rows, p.lens, p.refs = [[1, 2], [3, 5], [4]], [20, 17, 5], [0, 1, 1, 1, 1, 1] + [0] * 14
    p.up()
    p.t[1, 1] = entry
    out, lens = torch.full((len(parents), 4), 9, dtype=torch.int32, device=DEV), ints([9] * len(parents))
    dash.pages_fork(p.t, p.l, ints(parents), out, lens, p.c, 16)
    assert dash.get_status_paged() == (dash.ERR_PAGE, [4, 1, entry, 20])
    no_error()
    old = [[1, 2, -1, -1], [3, entry, -1, -1], [4, -1, -1, -1], [-1] * 4]
    assert out.tolist() == [old[q] for q in parents] and lens.tolist() == [[20, 17, 5, 0][q] for q in parents]
    children = [parents.count(r) for r in range(3)]
    want = list(p.refs)
    for r, row in enumerate(p.rows):
        for q in row:
            want[q] = children[r] if q != 5 else 1      # (the page that the bad entry stands for is not counted)
    assert p.c.tolist() == want


MOST = 2 ** 31 - 1   # rows and tokens are ints


def test_as_many_tokens_as_an_int_counts():
    """Three rows' tokens and padding to the end: counters do not pass 2^31."""
    p = Pool(random.Random(9), 20, 16, 4, 3, 30)
    n_new = [3, 1, 9]
    slots, pos = torch.full((MOST,), 7, dtype=torch.int64, device=DEV), torch.full((MOST,), 7, dtype=torch.int32, device=DEV)
    copies, counts = ints([[MARK] * 2] * 3), ints([MARK, MARK])
    dash.pages_extend(p.t, p.l, p.c, 16, slots, pos, copies, counts, cu_new=ints([0, 3, 4, 13]))
    p.rows, p.lens, p.refs, want, taken, at, where = PG.extend(p.rows, p.lens, p.refs, n_new, 16)
    assert counts.tolist() == [len(want), taken] and slots[:13].tolist() == where and pos[:13].tolist() == at
    assert int(slots[13:].max()) == int(slots[13:].min()) == -1 and int(pos[13:].max()) == int(pos[13:].min()) == 0
    p.check()
    no_error()


def test_as_many_rows_as_an_int_counts():
    """Forked from one row, and compacted: the first and the last hold a page, the others nothing."""
    parents = torch.full((MOST,), -1, dtype=torch.int32, device=DEV)
    parents[0] = parents[-1] = 0
    table, lens = torch.full((MOST, 1), 9, dtype=torch.int32, device=DEV), torch.full((MOST,), 9, dtype=torch.int32, device=DEV)
    refs = ints([1, 0, 0, 0, 0, 1])
    dash.pages_fork(ints([[5]]), ints([16]), parents, table, lens, refs, 16)
    assert table[0].tolist() == table[-1].tolist() == [5] and lens[0] == lens[-1] == 16 and refs.tolist() == [1, 0, 0, 0, 0, 2]
    assert int(table[1:-1].max()) == int(table[1:-1].min()) == -1 and int(lens[1:-1].max()) == int(lens[1:-1].min()) == 0
    copies, counts = ints([[MARK] * 2] * 3), ints([MARK, MARK])
    dash.pages_compact(table, lens, refs, 16, copies, counts)
    assert counts.tolist() == [1, 2] and copies.tolist() == [[5, 1]] + [[MARK] * 2] * 2 and refs.tolist() == [1, 2, 0, 0, 0, 0]
    assert table[0].tolist() == table[-1].tolist() == [1] and int(table[1:-1].max()) == int(table[1:-1].min()) == -1
    no_error()
