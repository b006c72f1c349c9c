"""The calls for pages without a GPU: every refusal that needs no device, and the plain forms themselves."""
import ctypes
import os
import random

import pytest
import torch

from oracle import pages as PG
from tile_scheduling_persistent_gb300 import dash

OK, BAD = 4096, 4098   # an aligned and a misaligned address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dash.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dash.lib()


def fork(L, table=OK, stride=8, lens=OK, rows=3, parents=OK, out=2 * OK, out_stride=8, lens_out=2 * OK, rows_out=4, width=8, refs=OK, N=10,
         page=16):
    return L.dash_pages_fork(table, stride, lens, rows, parents, out, out_stride, lens_out, rows_out, width, refs, N, page, None)


def extend(L, table=OK, stride=8, lens=OK, rows=3, width=8, refs=OK, N=10, page=16, cu=OK, slots=OK, positions=OK, T=6, copies=OK, counts=OK):
    return L.dash_pages_extend(table, stride, lens, rows, width, refs, N, page, cu, slots, positions, T, copies, counts, None)


def compact(L, table=OK, stride=8, lens=OK, rows=3, width=8, refs=OK, N=10, page=16, out=OK, out_stride=8, refs_out=OK, copies=OK, counts=OK,
            ws=OK, wn=40):
    return L.dash_pages_compact(table, stride, lens, rows, width, refs, N, page, out, out_stride, refs_out, copies, counts, ws, wn, None)


POOL = [dict(table=None), dict(table=BAD + 1), dict(stride=7), dict(stride=-8), dict(lens=None), dict(lens=BAD + 1), dict(rows=-1),
        dict(width=-1), dict(refs=None), dict(refs=BAD), dict(N=0), dict(N=-1), dict(N=(1 << 30) + 1), dict(page=8), dict(page=24), dict(page=512),
        dict(width=1 << 28, stride=1 << 28)]


@pytest.mark.parametrize("kw", POOL + [dict(parents=None), dict(parents=BAD + 1), dict(out=None), dict(out_stride=7), dict(lens_out=None),
                                       dict(rows_out=-1), dict(out=OK), dict(lens_out=OK)])
def test_fork_refuses(L, kw):
    assert fork(L, **kw) == dash.ERR_ARG


@pytest.mark.parametrize("kw", POOL + [dict(rows=4097), dict(cu=BAD + 1), dict(slots=None), dict(slots=BAD + 2), dict(positions=None),
                                       dict(positions=BAD + 1), dict(T=-1), dict(copies=None), dict(copies=BAD + 1), dict(counts=None),
                                       dict(counts=BAD + 1), dict(cu=None, T=7), dict(cu=None, rows=0, T=1)])
def test_extend_refuses(L, kw):
    assert extend(L, **kw) == dash.ERR_ARG


@pytest.mark.parametrize("kw", POOL + [dict(out=None), dict(out_stride=9), dict(refs_out=None), dict(refs_out=BAD), dict(copies=None),
                                       dict(counts=None), dict(ws=None), dict(ws=BAD)])
def test_compact_refuses(L, kw):
    assert compact(L, **kw) == dash.ERR_ARG


def test_compact_refuses_a_small_workspace(L):
    assert compact(L, wn=39) == dash.ERR_SCRATCH


def caches(n=2, **kw):
    at = dict(k=OK, v=OK, ks=0, vs=0, typ=0, pages=4, page=16, H=2, D=64)
    at.update(kw)
    one = lambda **k: dash._CACHE.pack(*{**at, **k}.values())  # noqa: E731
    return [one() for _ in range(n)], one


def copy(L, packed, n=None, copies=OK, count=OK, most=3):
    return L.dash_kv_copy(b"".join(packed) if packed is not None else None, len(packed or ()) if n is None else n, copies, count, most, None)


def test_copy_refuses(L):
    good, one = caches()
    for bad in (one(typ=1), one(pages=5), one(page=32), one(H=3), one(D=128), one(k=0), one(v=BAD), one(ks=OK), one(typ=1, ks=OK, vs=OK)):
        assert copy(L, good + [bad]) == dash.ERR_ARG
    assert copy(L, good, n=-1) == dash.ERR_ARG and copy(L, None, n=1) == dash.ERR_ARG
    assert copy(L, good, copies=None) == dash.ERR_ARG and copy(L, good, copies=BAD + 1) == dash.ERR_ARG
    assert copy(L, good, count=BAD + 1) == dash.ERR_ARG and copy(L, good, most=-1) == dash.ERR_ARG


def test_empty_calls_do_nothing(L):
    assert fork(L, rows=0, rows_out=0, table=None, lens=None, out=None, lens_out=None, parents=None) == dash.OK
    good, _ = caches()
    assert copy(L, []) == dash.OK and copy(L, good, most=0, copies=None) == dash.OK


def test_plain_forms_keep_every_rows_tokens():
    """Cells of the plain pool carry the tokens written into them: after any steps each row reads back its own tokens, refs
    are the table's counts, and nothing is lost or shared that should not be."""
    rng = random.Random(1)
    page, N = 4, 60
    cells = [[None] * page for _ in range(N)]
    table, lens, refs, text, token = [[]], [0], [0] * N, [[]], 0
    for step in range(400):
        kind = rng.randrange(5)
        if kind == 0:
            parents = [rng.choice([-1, rng.randrange(len(table))]) for _ in range(rng.randint(1, 6))]
            table, lens, refs = PG.fork(table, lens, parents, refs)
            text = [list(text[p]) if p >= 0 else [] for p in parents]
        elif kind == 1:
            table, refs, moves, live = PG.compact(table, refs)
            old = [list(c) for c in cells]
            for a, b in moves:
                cells[b] = old[a]
            assert all(r == 0 for r in refs[live:]) and all(r > 0 for r in refs[:live])
        else:
            new = [rng.randint(0, 6) for _ in table]
            got = PG.extend(table, lens, refs, new, page)
            if got is None:
                continue
            table, lens, refs, copies, taken, at, slots = got
            for a, b in copies:
                cells[b] = list(cells[a])
            where = iter(zip(at, slots))
            for r, n in enumerate(new):
                for _ in range(n):
                    pos, slot = next(where)
                    assert pos == len(text[r])
                    cells[slot // page][slot % page] = token
                    text[r].append(token)
                    token += 1
        count = [0] * N
        for r, row in enumerate(table):
            assert len(row) == PG.pages_of(lens[r], page) and len(text[r]) == lens[r]
            assert [cells[row[i // page]][i % page] for i in range(lens[r])] == text[r]
            for p in row:
                count[p] += 1
        assert count == refs


def test_the_binding_refuses_what_the_library_cannot_see(L, monkeypatch):
    monkeypatch.setattr(dash, "_device_stream", lambda stream, what: (-1, 0))   # (CPU tensors stand for the device's)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    table, lens, refs = i32(3, 8), i32(3), i32(12)
    for kw in (dict(table=i32(3, 8).long()), dict(table=i32(2, 8)), dict(lens=i32(3, 1)), dict(refs=i32(12).long()), dict(parents=i32(5)),
               dict(table_out=i32(4, 7)), dict(lens_out=i32(5)), dict(table=i32(1, 8).expand(3, 8)), dict(table=i32(8, 3).t())):
        at = {**dict(table=table, lens=lens, parents=i32(4), table_out=i32(4, 8), lens_out=i32(4), refs=refs), **kw}
        with pytest.raises(dash.DashError):
            dash.pages_fork(*at.values(), 16)
    for kw in (dict(slots=i32(6)), dict(positions=i32(5)), dict(copies=i32(3, 3)), dict(copies=i32(2, 2)), dict(counts=i32(3)), dict(cu_new=i32(3))):
        at = {**dict(slots=i32(6).long(), positions=i32(6), copies=i32(3, 2), counts=i32(2), cu_new=i32(4)), **kw}
        with pytest.raises(dash.DashError):
            dash.pages_extend(table, lens, refs, 16, **at)
    for kw in (dict(copies=i32(5, 2)), dict(counts=i32(1)), dict(table_out=i32(3, 9)), dict(refs_out=i32(13)), dict(workspace=i32(12))):
        at = {**dict(copies=i32(6, 2), counts=i32(2), workspace=torch.zeros(48, dtype=torch.uint8)), **kw}
        with pytest.raises(dash.DashError):
            dash.pages_compact(table, lens, refs, 16, **at)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for a in (([k], [k, k], i32(1, 2)), ([k], [k], i32(1, 3)), ([k], [k], i32(2)), ([k], [k.float()], i32(1, 2)), ([k], [k], i32(1, 2).long())):
        with pytest.raises(dash.DashError):
            dash.kv_copy(*a)
    with pytest.raises(dash.DashError):
        dash.kv_copy([k], [k], i32(1, 2), k_scales=[i32(1)], v_scales=[])


@pytest.mark.parametrize("rows,rows_out", [(2 ** 20 + 1, 2 ** 20), (2 ** 31 - 1, 2 ** 31 - 1), (513, 2 ** 31 - 1)])
def test_fork_refuses_more_pairs_of_rows_than_it_can_look_at(L, rows, rows_out):
    assert fork(L, rows=rows, rows_out=rows_out, width=0, stride=0, out_stride=0) == dash.ERR_ARG
