"""A cache of 4 bits used as a server uses it: prompts written, forked, decoded in branches, some dropped, the pool compacted,
and decoding again -- every token's attention against a plain run that keeps each row's own keys and values."""
import random

import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from cache4_helpers import quantised4, values4
from serving_helpers import DEV, E4M3, no_error, paged, randn

pytestmark = pytest.mark.gpu


class Server:
    """Two layers over one pool; `text` holds each row's keys and values as the cache has them, in 64 bits."""

    def __init__(self, kind, Hq, Hkv, D, page, pages, width, seed):
        self.g, self.kind, self.Hq, self.Hkv, self.D, self.page = torch.Generator().manual_seed(seed), kind, Hq, Hkv, D, page
        shape = (pages, Hkv, page)
        made = lambda last, mark: torch.full(shape + (last,), mark, dtype=torch.uint8, device=DEV)  # noqa: E731
        if kind == "e2m1":
            self.k, self.v = ([made(D // 2, 0xff) for _ in range(2)] for _ in range(2))
            self.ks, self.vs = ([made(D // 16, 0x7f).view(E4M3) for _ in range(2)] for _ in range(2))
            self.exps = dict(k_exp=-3, v_exp=-2)
        else:
            self.k, self.v = ([torch.full(shape + (D,), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(2))
            self.ks = self.vs = None
            self.exps = {}
        self.table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
        self.lens, self.refs = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.text = [[[np.zeros((0, Hkv, D)) for _ in range(2)] for _ in range(2)]]   # [row][layer][k, v]

    def scales(self, layer):
        return dict(k_scale=self.ks[layer], v_scale=self.vs[layer], **self.exps) if self.ks else {}

    def copy(self, copies, counts):
        dash.kv_copy(self.k, self.v, copies, counts, **(dict(k_scales=self.ks, v_scales=self.vs) if self.ks else {}))

    def fork(self, parents):
        t = torch.full((len(parents), self.table.shape[1]), 77, dtype=torch.int32, device=DEV)
        n = torch.zeros(len(parents), dtype=torch.int32, device=DEV)
        dash.pages_fork(self.table, self.lens, torch.tensor(parents, dtype=torch.int32, device=DEV), t, n, self.refs, self.page)
        self.table, self.lens = t, n
        empty = np.zeros((0, self.Hkv, self.D))
        self.text = [[list(x) for x in self.text[p]] if p >= 0 else [[empty, empty], [empty, empty]] for p in parents]

    def compact(self):
        copies = torch.zeros(self.refs.shape[0] // 2, 2, dtype=torch.int32, device=DEV)
        counts = torch.zeros(2, dtype=torch.int32, device=DEV)
        dash.pages_compact(self.table, self.lens, self.refs, self.page, copies, counts)
        self.copy(copies, counts)
        return int(counts[0])

    def held(self, x, exp):
        if self.kind != "e2m1":
            return x.double().numpy()
        return values4(*quantised4(x, exp), exp).numpy()

    def step(self, n_new, pad=2):
        """New tokens of every row: written and attended to in both layers, and checked."""
        R, T = len(n_new), sum(n_new) + pad
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n_new)]), dtype=torch.int32, device=DEV)
        slots, pos = torch.zeros(T, dtype=torch.int64, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
        copies, counts = torch.zeros(R, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
        dash.pages_extend(self.table, self.lens, self.refs, self.page, slots, pos, copies, counts, cu_new=cu)
        self.copy(copies, counts)
        for layer in range(2):
            qkv = randn(self.g, T, self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.to(DEV).split([self.Hq, self.Hkv, self.Hkv], dim=1)
            dash.kv_write(k, v, self.k[layer], self.v[layer], slots, **self.scales(layer))
            o = torch.full((T, self.Hq, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
            dash.attn_paged(q, self.k[layer], self.v[layer], self.table, self.lens, o, cu_q=cu, max_q=max(max(n_new), 1), **self.scales(layer))
            no_error()
            o = o.float().cpu().double().numpy()
            at = 0
            for r, n in enumerate(n_new):
                hq = qkv[at:at + n]
                for x, (heads, exp) in enumerate(((slice(self.Hq, self.Hq + self.Hkv), -3), (slice(self.Hq + self.Hkv, None), -2))):
                    self.text[r][layer][x] = np.concatenate([self.text[r][layer][x], self.held(hq[:, heads], exp)])
                kk, vv = self.text[r][layer]
                rows = hq[:, :self.Hq].double().numpy()
                ro, _ = V.attend(rows, kk, vv, kk.shape[0] - n)
                A, _ = V.attend(rows, kk, np.abs(vv), kk.shape[0] - n)
                # (serving_helpers.check_attn's bound, which has room for either cache)
                assert (np.abs(o[at:at + n] - ro) <= (2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -8 * np.abs(ro)).all(), (r, layer)
                at += n
            assert (o[at:] == 77.0).all()
        assert self.lens.cpu().tolist() == [t[0][0].shape[0] for t in self.text]
        count = torch.zeros_like(self.refs.cpu())
        for r, t in enumerate(self.text):
            for p in self.table[r, :-(-t[0][0].shape[0] // self.page)].cpu().tolist():
                count[p] += 1
        assert torch.equal(count, self.refs.cpu())


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (4, 4, 64, 32)])
def test_a_servers_steps(kind, Hq, Hkv, D, page):
    s = Server(kind, Hq, Hkv, D, page, pages=90, width=20, seed=3)
    s.fork([0, 0, 0])
    s.step([75, 130, 16])                 # three prompts
    s.fork([0, 0, 0, 1, 2, 2, -1])        # branches, and a row that is still empty
    s.step([1, 1, 1, 1, 1, 1, 3])
    s.step([5, 1, 0, 3, 1, 2, 1])
    s.fork([1, 3, 5, 6, 5])               # a beam's step: some dropped, one doubled
    s.step([1, 1, 1, 1, 1])
    assert s.compact() > 0
    s.step([1, 2, 1, 40, 1])
    s.fork([4, -1])
    s.compact()
    s.step([9, 21])


def test_random_service():
    rng = random.Random(5)
    s = Server("e2m1", 6, 2, 64, 16, pages=120, width=12, seed=9)
    s.fork([0, 0])
    s.step([50, 7])
    for step in range(12):
        rows = len(s.text)
        if step % 3 == 0:
            s.fork([rng.choice([i, rng.randrange(rows)]) if i < rows else rng.randrange(-1, rows) for i in range(rng.randint(2, 6))])
        elif step % 3 == 1:
            s.compact()
        s.step([min(rng.choice([0, 1, 1, 2, 18]), 12 * 16 - t[0][0].shape[0]) for t in s.text], pad=rng.choice([0, 1]))
