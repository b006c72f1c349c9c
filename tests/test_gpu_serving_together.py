"""Rotary positions, the paged cache and its attention used together, as a server and a training step use them, and
calls at the edges of what is documented."""
import threading

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from gpu_helpers import check
from serving_helpers import DEV, E4M3, Paged, check_attn, no_error, paged, randn, raw, rope_bound, run_attn, same

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Server:
    """A cache and the per-step calls of one attention layer: rotate and write the new tokens, then attend."""

    def __init__(self, B, longest, Hq, Hkv, D, page, quant, seed):
        g = gen(seed)
        width = -(-longest // page)
        N = B * width + 1
        self.Hq, self.Hkv, self.D, self.page = Hq, Hkv, D, page
        self.table = torch.randperm(N, generator=g)[:B * width].reshape(B, width).to(torch.int32)
        shape = (N, Hkv, page, D)
        if quant:
            self.k, self.v = (torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
            self.kw = dict(k_scale=torch.full(shape[:3], float("nan"), device=DEV), v_scale=torch.full(shape[:3], float("nan"), device=DEV))
        else:
            self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            self.kw = {}
        self.table_dev = self.table.to(DEV)
        self.lens = [0] * B
        self.freqs, self.factor = dash.rope_freqs(D, 500000.0, "wave", scale=8.0, trained=8192, lo=1.0, hi=4.0)

    def places(self, n):
        """Slots and positions of n[b] new tokens each, packed."""
        pos = np.concatenate([np.arange(ln, ln + m) for ln, m in zip(self.lens, n)])
        seq = np.repeat(np.arange(len(n)), n)
        slot = self.table.numpy()[seq, pos // self.page].astype(np.int64) * self.page + pos % self.page
        return torch.from_numpy(slot), torch.from_numpy(pos.astype(np.int32))

    def call(self, qkv, slots, positions, cu, lens, o, lse, max_q):
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=1)   # one projection's rows
        dash.kv_write(k, v, self.k, self.v, slots, inv_freq=self.freqs, positions=positions, factor=self.factor, q=q, q_out=q, **self.kw)
        dash.attn_paged(q, self.k, self.v, self.table_dev, lens, o, cu_q=cu, max_q=max_q, lse=lse, **self.kw)

    def step(self, qkv, n):
        slots, positions = self.places(n)
        self.lens = [ln + m for ln, m in zip(self.lens, n)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        o = torch.full((sum(n), self.Hq, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((sum(n), self.Hq), 77.0, device=DEV)
        x = qkv.to(DEV)
        self.call(x, slots.to(DEV), positions.to(DEV), cu, torch.tensor(self.lens, dtype=torch.int32, device=DEV), o, lse, max(n))
        return x[:, :self.Hq], o, lse

    def held(self):
        """What the cache stands for, [len, Hkv, D] of each sequence, in 64 bits."""
        out = []
        for pages, scale in ((self.k, self.kw.get("k_scale")), (self.v, self.kw.get("v_scale"))):
            x = pages.float().cpu().double().numpy()
            if scale is not None:
                x = x * scale.cpu().double().numpy()[..., None]
            out.append([x[self.table[b].long().numpy()].transpose(0, 2, 1, 3).reshape(-1, self.Hkv, self.D)[:ln]
                        for b, ln in enumerate(self.lens)])
        return out

    def state(self):
        k, v = self.held()
        return Paged(k, v, self.k, self.v, self.kw.get("k_scale"), self.kw.get("v_scale"), self.table_dev,
                     torch.tensor(self.lens, dtype=torch.int32, device=DEV), self.kw)


@pytest.mark.parametrize("quant", [False, True])
def test_prompts_in_chunks_drafts_and_replayed_decoding(quant):
    # Two sequences grow to 256 tokens: prompts in two chunks, a few drafted tokens, then single tokens from a captured
    # step.  Every token's output, collected over the steps, is causal attention over the whole sequence.
    Hq, Hkv, D = 8, 2, 128
    s = Server(2, 256, Hq, Hkv, D, 16, quant, 21)
    x = [randn(gen(22 + b), 256, Hq + 2 * Hkv, D) for b in range(2)]
    got = [[[], [], []], [[], [], []]]   # of each sequence: rotated queries, o, lse

    def take(n, parts):
        at = 0
        for b, m in enumerate(n):
            for i in range(3):
                got[b][i].append(parts[i][at:at + m].clone())
            at += m

    for n in ([150, 37], [96, 210], [5, 4]):
        now = torch.cat([x[b][s.lens[b]:s.lens[b] + m] for b, m in enumerate(n)])
        take(n, s.step(now, n))
    take([1, 1], s.step(torch.stack([x[b][s.lens[b]] for b in range(2)]), [1, 1]))
    no_error()
    # a decoding step, captured once and replayed for each token
    qkv = torch.empty(2, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    slots, pos = torch.empty(2, dtype=torch.int64, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    lens = torch.empty(2, dtype=torch.int32, device=DEV)
    o, lse = torch.empty(2, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(2, Hq, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call(qkv, slots, pos, None, lens, o, lse, 1)
    for _ in range(4):
        qkv.copy_(torch.stack([x[b][s.lens[b]] for b in range(2)]))
        sl, p = s.places([1, 1])
        slots.copy_(sl)
        pos.copy_(p)
        s.lens = [ln + 1 for ln in s.lens]
        lens.copy_(torch.tensor(s.lens, dtype=torch.int32))
        graph.replay()
        take([1, 1], (qkv[:, :Hq], o, lse))
    no_error()
    assert s.lens == [256, 256]
    q, o, lse = (torch.cat([torch.cat(got[b][i]) for b in range(2)]) for i in range(3))
    check_attn(s.state(), q.cpu(), [256, 256], o, lse)
    # the rotated queries, and the keys as the cache returns them
    k, v = (torch.full((2, Hkv, 256, D), 77.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dash.kv_read(s.k, s.v, s.table_dev, torch.tensor(s.lens, dtype=torch.int32, device=DEV), k, v, **s.kw)
    no_error()
    f = s.freqs.numpy()
    for b in range(2):
        xb = x[b].double().numpy()
        pos = np.arange(256)[:, None]
        ref = V.rope(xb[:, :Hq], pos, f, s.factor)
        assert (np.abs(q[256 * b:256 * (b + 1)].double().cpu().numpy() - ref) <= rope_bound(xb[:, :Hq], f, s.factor, False, True, ref)).all()
        ref = V.rope(xb[:, Hq:Hq + Hkv], pos, f, s.factor).transpose(1, 0, 2)
        d = np.abs(k[b].double().cpu().numpy() - ref)
        bound = rope_bound(xb[:, Hq:Hq + Hkv].transpose(1, 0, 2), f, s.factor, False, True, ref)
        if quant:   # codes: half a step, 2^-4 of the value, and 2^-10 of the scale below the least normal code
            bound = bound + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * np.abs(ref).max(-1, keepdims=True) / 448 * 1.01
        assert (d <= bound * 1.01).all()
        if not quant:
            assert same(v[b].cpu(), x[b][:, Hq + Hkv:].transpose(0, 1).contiguous())
    # the contiguous kernel over what the cache returned
    oc = torch.empty(2, Hq, 256, D, dtype=torch.bfloat16, device=DEV)
    lc = torch.empty(2, Hq, 256, device=DEV)
    qc = q.reshape(2, 256, Hq, D).transpose(1, 2).contiguous()
    dash.attn_fwd(qc, k, v, oc, lc, True)
    ref, _ = A.attn_fwd(qc.cpu(), k.cpu(), v.cpu(), True)
    check("attn_fwd over the cache's keys and values", oc, ref)


@pytest.mark.parametrize("inter", [False, True])
def test_a_training_step_through_rotated_attention(inter):
    # Forward: rotate, attend.  Backward: the attention's, then the inverse rotation of dQ from its fp32 accumulator and
    # of dK.  Against the 64-bit formula, and along a direction against differences of the 64-bit forward.
    B, Hq, Hkv, S, D = 1, 4, 2, 256, 64
    f, _ = dash.rope_freqs(D, 10000.0)
    q, k, v, do = (randn(gen(30 + i), B, h, S, D) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    dev = [t.to(DEV) for t in (q, k, v, do)]
    qr, kr = torch.empty_like(dev[0]), torch.empty_like(dev[1])
    o, lse = torch.empty_like(dev[0]), torch.empty(B, Hq, S, device=DEV)
    acc, dkr, dv = torch.empty(B, Hq, S, D, device=DEV), torch.empty_like(dev[1]), torch.empty_like(dev[2])
    dq, dk = torch.empty_like(dev[0]), torch.empty_like(dev[1])
    dash.rope(dev[0], qr, f, x2=dev[1], y2=kr, interleaved=inter)
    dash.attn_fwd(qr, kr, dev[2], o, lse, True)
    dash.attn_bwd(qr, kr, dev[2], o, dev[3], lse, acc, dkr, dv, True, "auto")
    dash.rope(acc, dq, f, x2=dkr, y2=dk, interleaved=inter, inverse=True)
    assert dash.get_status()[0] == 0
    pos, fn = np.arange(S), f.numpy()
    # the inverse rotation, element by element
    for got, x in ((dq, acc), (dk, dkr)):
        xn = x.double().cpu().numpy()
        ref = V.rope(xn, pos, fn, 1.0, inter, inverse=True)
        assert (np.abs(got.double().cpu().numpy() - ref) <= rope_bound(xn, fn, 1.0, inter, True, ref)).all()
    # The step against the formula in 64 bits from the unrounded rotation.  Norms: q and k are off by at most 2^-8 of
    # themselves (rounded after the rotation), so scores by 2 * 2^-8 |q| |k| / 8 <= 2^-7 * 13 * 13 / 8 = 0.17 at the very worst;
    # rounding errors are independent, uniform within half a step (rms 2^-8 / sqrt(3) of the step's upper end, 0.6 of that on
    # average over a binade), so a score's 2 * 64 errors add to about sqrt(2 * 64) * 2^-8 * 0.35 / 8 = 1.9e-3, and
    # weights, their gradients, o and do's products take the same relative error a few times over: within 2e-2 of the norm.
    q64, k64, v64, do64 = (t.double().numpy() for t in (q, k, v, do))

    def forward(a, b):
        return A.attn_fwd(V.rope(a, pos, fn, 1.0, inter), V.rope(b, pos, fn, 1.0, inter), v64, True)

    ro, rlse = forward(q64, k64)
    rdq, rdk, rdv, _ = A.attn_bwd(V.rope(q64, pos, fn, 1.0, inter), V.rope(k64, pos, fn, 1.0, inter), v64, ro, do64, rlse, True)
    rdq, rdk = V.rope(rdq, pos, fn, 1.0, inter, inverse=True), V.rope(rdk, pos, fn, 1.0, inter, inverse=True)
    for got, ref in ((dq, rdq), (dk, rdk), (dv, rdv)):
        assert np.linalg.norm(got.double().cpu().numpy() - ref) <= 2e-2 * np.linalg.norm(ref)
    # Differences: central, h = 1e-4 (error h^2 times third derivatives of order one; fp64 leaves 1e-11 / h), along the
    # gradient itself, where the kernels' gradient g is within 2e-2 |ref| of ref, hence <g, ref> within 2e-2 of |ref|^2.
    h = 1e-4
    norm = float((rdq ** 2).sum() + (rdk ** 2).sum()) ** 0.5
    up, down = (forward(q64 + t * rdq / norm, k64 + t * rdk / norm)[0] for t in (h, -h))
    slope = float((do64 * (up - down)).sum()) / (2 * h)
    mine = (float((dq.double().cpu().numpy() * rdq).sum()) + float((dk.double().cpu().numpy() * rdk).sum())) / norm
    assert abs(slope - norm) <= 1e-4 * norm and abs(mine - slope) <= 2.1e-2 * norm


@pytest.mark.parametrize("quant", [False, True])
def test_more_sequences_than_one_launch_holds(quant):
    g = gen(40)
    B = 1100
    lens = [3000 if i % 300 == 7 else 1 + 37 * i % 200 for i in range(B)]
    n = [min(40, lens[i]) if i % 90 == 3 else 0 if i % 50 == 9 else 1 for i in range(B)]
    c = paged(g, lens, 2, 64, 16, quant)
    q = randn(g, sum(n) + 2, 8, 64)
    o, lse = run_attn(c, q, n)
    no_error()
    check_attn(c, q, n, o, lse)


@pytest.mark.parametrize("Hq,Hkv,n", [(320, 320, [1, 1]), (320, 320, [20, 3]), (34, 2, [1, 2]), (34, 2, [40, 9]), (100, 1, [1, 30])])
@pytest.mark.parametrize("quant", [False, True])
def test_many_heads_and_odd_groups(Hq, Hkv, n, quant):
    g = gen(41)
    c = paged(g, [70, 700], Hkv, 64, 32, quant)
    q = randn(g, sum(n), Hq, 64)
    o, lse = run_attn(c, q, n)
    no_error()
    check_attn(c, q, n, o, lse)


@pytest.mark.parametrize("n", [[1, 1, 1], [2, 2, 1], [200, 30, 1]])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(n, D):
    # e4m3: neighbouring tokens' scales differ by up to 2^16, and grow by 2^3 with every 128 keys; some vectors are zero (least
    # scale, zero codes) or have a scale of zero.  Products with a power of two are exact, so check_attn's bound holds as
    # it is: values are held to 2^-11 of themselves and 2^-31 of the largest, far below its 2^-8 A within 2^16.
    g = gen(42)
    c = paged(g, [700, 300, 1], 2, D, 16, True)
    for b, ln in enumerate([700, 300, 1]):
        kp, vp = torch.randint(-3, 1, (ln, 2), generator=g), torch.randint(-8, 9, (ln, 2), generator=g)
        vp = vp + (3 * (torch.arange(ln) // 128))[:, None]
        j = torch.arange(ln)
        p, at = c.table[b].cpu().long()[j // 16], j % 16
        kf, vf = torch.exp2(kp.float()), torch.exp2(vp.float())
        if ln > 9:
            kf[4], vf[5], vf[9] = 0.0, 0.0, 0.0
        else:
            vf[0] = 0.0
        for scale, f, held in ((c.k_scale, kf, c.k), (c.v_scale, vf, c.v)):
            host = scale.cpu()
            host[p, :, at] *= f
            scale.copy_(host)
            held[b] *= f.double().numpy()[..., None]
        if ln > 9:   # a zero vector as kv_write leaves it
            raw(c.v_cache)[p[9], :, at[9]] = 0
            c.v_scale[p[9], :, at[9]] = 2.0 ** -126
    q = randn(g, sum(n), 8, D)
    o, lse = run_attn(c, q, n)
    no_error()
    check_attn(c, q, n, o, lse)


@pytest.mark.parametrize("n", [[1, 1], [2, 1], [50, 70]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [False, True])
def test_queries_that_are_not_finite_stay_in_their_rows(n, D, quant):
    g = gen(43)
    c = paged(g, [5000, 200], 2, D, 16, quant)   # one split into key ranges, one not
    q = randn(g, sum(n), 8, D)
    bad = [(0, 1), (0, 6), (sum(n) - 1, 3)]
    d = q.clone()
    for (t, h), x in zip(bad, (float("nan"), float("inf"), -float("inf"))):
        d[t, h, 5] = x
    o, lse = run_attn(c, d, n)
    no_error()
    clean, clse = run_attn(c, q, n)
    for t, h in bad:
        assert bool(torch.isnan(o[t, h]).any()) and bool(torch.isnan(lse[t, h]))   # as the formula has it
        o[t, h], lse[t, h] = clean[t, h], clse[t, h]
    check_attn(c, q, n, o, lse)


def test_two_graphs_share_a_workspace():
    # one after the other on a stream: each replay finds what the other left there
    g = gen(44)
    c = paged(g, [3000, 900, 2000], 2, 128, 16, True)
    calls = []
    for n in ([1, 1, 1], [2, 150, 40]):
        q = randn(g, sum(n), 16, 128).to(DEV)
        ref = run_attn(c, q, n)[0]
        calls.append((q, torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV), max(n), ref, torch.empty_like(q)))
    ws = torch.full((max(dash.attn_paged_workspace(3, q.shape[0], 16, 2, 128, m, c.table.shape[1] * 16) for q, _, m, _, _ in calls),), 0xff,
                    dtype=torch.uint8, device=DEV)
    graphs = []
    for q, cu, m, _, o in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=m, workspace=ws, **c.kw)
        graphs.append(graph)
    for i in (0, 1, 0, 0, 1, 1, 0, 1):
        calls[i][4].fill_(77.0)
        graphs[i].replay()
        assert same(calls[i][4], calls[i][3])
    no_error()


def test_the_bindings_own_workspace():
    # threads on one stream, streams of one thread, and a replayed graph beside eager calls, all without a workspace of
    # the caller's: nobody finds another's partial results in its own
    c = paged(gen(50), [3000, 900, 2000], 2, 128, 16, True)
    work = []
    for n in ([1, 1, 1], [2, 150, 40], [3, 3, 9]):
        q = randn(gen(51), sum(n), 16, 128).to(DEV)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        work.append((q, cu, max(n), run_attn(c, q, n)[0]))
    torch.cuda.synchronize()

    def call(i, o):
        q, cu, m, _ = work[i]
        dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=m, **c.kw)

    wrong = []

    def thread(first):
        outs = []
        for k in range(30):
            i = (first + k) % 3
            outs.append((i, torch.full_like(work[i][0], 77.0)))
            call(*outs[-1])
        torch.cuda.synchronize()
        wrong.extend(i for i, o in outs if not same(o, work[i][3]))

    threads = [threading.Thread(target=thread, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    captured = torch.empty_like(work[1][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(1, captured)
    side, eager = torch.cuda.Stream(), []
    for k in range(20):
        captured.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        for i in range(3):
            eager.append((i, torch.full_like(work[i][0], 77.0)))
            call(*eager[-1])
        torch.cuda.current_stream().wait_stream(side)
        assert same(captured, work[1][3])
    assert all(same(o, work[i][3]) for i, o in eager)
    no_error()
    dash.release_workspaces()
    call(1, captured)
    assert same(captured, work[1][3])


@pytest.mark.parametrize("n", [[1, 1], [0, 60]])
def test_tables_without_pages(n):
    q = randn(gen(45), sum(n), 8, 64).to(DEV)
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    o = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device=DEV)
    table = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    dash.attn_paged(q, pages, pages, table, zero, o, cu_q=cu, max_q=max(n), lse=lse)
    k = torch.full((2, 2, 8, 64), 77.0, dtype=torch.bfloat16, device=DEV)
    dash.kv_read(pages, pages, table, zero, k, k.clone())
    no_error()
    assert (o == 0).all() and (lse == -float("inf")).all() and (k == 77.0).all()


@pytest.mark.parametrize("cu", [[0, 2, 1, 3], [0, 60, 20, 80]])
def test_first_rows_that_decrease_are_reported(cu):
    c = paged(gen(46), [3000, 500, 3000], 2, 64, 16, False)
    T = cu[-1]
    q = randn(gen(47), T, 8, 64).to(DEV)
    o = torch.full((T + 30, 8, 64), 77.0, dtype=torch.bfloat16, device=DEV)
    dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o[:T], cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV), max_q=60)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info[:2] == [3, 1]
    assert (o[T:] == 77.0).all()


def test_queries_with_a_stride_of_zero_are_refused():
    c = paged(gen(48), [30, 40], 2, 64, 16, False)
    q = randn(gen(49), 2, 4, 64).to(DEV)
    for x in (q[:1].expand(2, 4, 64), q[:, :1].expand(2, 4, 64)):
        with pytest.raises(dash.DashError):
            dash.attn_paged(x, c.k_cache, c.v_cache, c.table, c.lens, torch.empty_like(q))
    # the writer may read broadcast keys and values
    k, v = torch.zeros_like(c.k_cache), torch.zeros_like(c.v_cache)
    slots = torch.tensor([5, 33], dtype=torch.int64, device=DEV)
    dash.kv_write(q[:, :1].expand(2, 2, 64), q[:1, :2].expand(2, 2, 64), k, v, slots)
    no_error()
    assert same(k[0, :, 5], q[0, :1].expand(2, 64).contiguous()) and same(v[2, :, 1], q[0, :2])
