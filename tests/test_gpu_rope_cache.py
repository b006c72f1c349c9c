"""Rotary positions, cache writing and reading on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

from serving_helpers import DEV, E4M3, no_error, paged, quantised, randn, raw, rope_bound, same

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


ROPES = [
    # B, H, H2, S, D, rot, interleaved, inverse, x fp32, y fp32
    (1, 1, 1, 1, 64, 64, False, False, False, False),
    (2, 4, 2, 33, 128, 128, False, False, False, False),
    (2, 3, 1, 7, 128, 64, True, False, False, False),
    (3, 2, 2, 100, 64, 32, True, True, True, False),
    (1, 5, 0, 257, 128, 96, False, True, True, True),
    (2, 2, 2, 50, 64, 16, False, False, False, True),
    (1, 32, 8, 300, 128, 16, True, True, False, False),
]


@pytest.mark.parametrize("case", ROPES)
@pytest.mark.parametrize("positions", ["none", "shared", "own", "far"])
def test_rope(case, positions):
    B, H, H2, S, D, rot, inter, inverse, x32, y32 = case
    g = gen(1)
    f, _ = dash.rope_freqs(rot, 10000.0)
    factor = 1.25 if inter else 1.0
    pos = {"none": None, "shared": torch.arange(S) * 3 + 5, "own": torch.randint(0, 9000, (B, S), generator=g),
           "far": torch.randint(2 ** 30, 2 ** 31 - 1, (B, S), generator=g) * torch.where(torch.rand(B, S, generator=g) < 0.3, -1, 1)}[positions]
    ref_pos = np.arange(S)[None] if pos is None else pos.numpy().reshape(-1, S)
    args, outs, refs = [], [], []
    for h in (H, H2):
        if h == 0:
            continue
        x = torch.randn(B, h, S, D, generator=g)
        x = x if x32 else x.to(torch.bfloat16)
        y = torch.full((B, h, S, D), 5.0, dtype=torch.float32 if y32 else torch.bfloat16, device=DEV)
        args.append(x)
        outs.append(y)
        refs.append(V.rope(x.double().numpy(), ref_pos[:, None], f.numpy(), factor, inter, inverse))
    two = dict(x2=args[1].to(DEV), y2=outs[1]) if H2 else {}
    dash.rope(args[0].to(DEV), outs[0], f, positions=None if pos is None else pos.to(torch.int32).to(DEV), interleaved=inter,
              factor=factor, inverse=inverse, **two)
    for x, y, ref in zip(args, outs, refs):
        d = np.abs(y.double().cpu().numpy() - ref)
        assert (d <= rope_bound(x.double().numpy(), f, factor, inter, not y32, ref)).all(), d.max()
        if rot < D:
            assert torch.equal(y[..., rot:].cpu().float(), x[..., rot:].to(y.dtype).float())


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_and_strided(inter):
    # queries and keys inside one projection's rows [B, S, (Hq + 2 Hkv) * D], rotated where they lie
    B, S, Hq, Hkv, D = 2, 45, 4, 2, 128
    f, _ = dash.rope_freqs(D, 500000.0)
    qkv = randn(gen(2), B, S, Hq + 2 * Hkv, D).to(DEV)
    before = qkv.clone()
    q, k, v = qkv.permute(0, 2, 1, 3).split([Hq, Hkv, Hkv], dim=1)
    qo, ko = torch.empty(B, Hq, S, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hkv, S, D, dtype=torch.bfloat16, device=DEV)
    dash.rope(q, qo, f, x2=k, y2=ko, interleaved=inter)
    dash.rope(q, q, f, x2=k, y2=k, interleaved=inter)
    assert same(q.contiguous(), qo) and same(k.contiguous(), ko)
    assert same(v.contiguous(), before.permute(0, 2, 1, 3)[:, Hq + Hkv:].contiguous())
    ref = V.rope(before.permute(0, 2, 1, 3)[:, :Hq].double().cpu().numpy(), np.arange(S), f.numpy(), 1.0, inter)
    d = np.abs(qo.double().cpu().numpy() - ref)
    assert (d <= rope_bound(before.permute(0, 2, 1, 3)[:, :Hq].double().cpu().numpy(), f, 1.0, inter, True, ref)).all()


def test_rope_backward_is_the_transpose():
    # <R x, g> = <x, R^T g>: both sides in fp32 outputs, summed in 64 bits
    f, factor = dash.rope_freqs(128, 10000.0, "ramp", scale=8.0, trained=4096, lo=1.0, hi=32.0)
    x, g = torch.randn(2, 3, 65, 128, generator=gen(3)).to(DEV), torch.randn(2, 3, 65, 128, generator=gen(4)).to(DEV)
    pos = torch.randint(0, 100000, (2, 65), generator=gen(5)).to(torch.int32).to(DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dash.rope(x, y, f, positions=pos, factor=factor)
    dash.rope(g, dx, f, positions=pos, factor=factor, inverse=True)
    a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    # every product is off by at most 2^-20 of the pair's absolute values: |error| <= 2 * 2^-20 * factor * sum (|x| + |x'|) |g|
    assert abs(float(a - b)) <= 4 * 2.0 ** -20 * factor * 2 * float((x.abs().double() * g.abs().double()).sum())


def test_rope_refuses_shapes():
    x = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    f, _ = dash.rope_freqs(64)
    bad = [dict(y=x[:, :1]), dict(y=x.half()), dict(positions=torch.zeros(7, dtype=torch.int32, device=DEV)),
           dict(positions=torch.zeros(8, dtype=torch.int64, device=DEV)), dict(x2=x), dict(y2=x), dict(x=x[0], y=x[0]),
           dict(x2=x[:, :, :4], y2=x[:, :, :4]), dict(y=x[:, :1].expand(2, 2, 8, 64)), dict(x=x.transpose(2, 3), y=x.transpose(2, 3)),
           dict(inv_freq=f.to(DEV)), dict(inv_freq=f.float()), dict(y=x.cpu())]
    for kw in bad:
        with pytest.raises(dash.DashError):
            dash.rope(**{**dict(x=x, y=torch.empty_like(x), inv_freq=f), **kw})
    dash.rope(x[:, :, :0], x[:, :, :0], f)


WRITES = [
    # T, Hq, Hkv, D, page, rot, interleaved
    (1, 4, 1, 64, 16, 64, False),
    (1, 32, 8, 128, 16, 128, False),
    (37, 6, 2, 128, 32, 64, True),
    (130, 8, 4, 64, 64, 32, True),
    (300, 3, 3, 128, 256, 128, False),
    (513, 0, 2, 128, 128, 0, False),
    (70, 0, 5, 64, 16, 48, False),
]


def write_case(case, quant, seed=6):
    T, Hq, Hkv, D, page, rot, inter = case
    g = gen(seed)
    qkv = randn(g, T, Hq + 2 * Hkv, D)
    if T > 5:
        qkv[3] = 0.0                       # zero vectors
        qkv[4, -1, 5] = float("nan")       # a NaN stays in its own value
        qkv[5] *= 2.0 ** 100               # large and tiny vectors
    if T > 7:
        qkv[6] *= 2.0 ** -120
    N = -(-T // page) + 2
    slots = torch.randperm(N * page, generator=g)[:T]
    if T > 2:
        slots[T // 2] = -1
        slots[T - 1] = -(2 ** 40)
    pos = torch.randint(0, 200000, (T,), generator=g)
    shape = (N, Hkv, page, D)
    if quant:
        caches = [torch.full(shape, 3, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
        scales = [torch.full(shape[:3], 9.0, device=DEV) for _ in range(2)]
    else:
        caches, scales = [torch.full(shape, 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)], [None, None]
    return qkv, slots, pos, caches, scales


@pytest.mark.parametrize("case", WRITES)
@pytest.mark.parametrize("quant", [False, True])
def test_write(case, quant):
    T, Hq, Hkv, D, page, rot, inter = case
    qkv, slots, pos, (kc, vc), (ks, vs) = write_case(case, quant)
    f, factor = (dash.rope_freqs(rot, 10000.0)[0], 1.0) if rot else (None, 1.0)
    dev = qkv.to(DEV)
    q, k, v = dev.split([Hq, Hkv, Hkv], dim=1)
    kw = dict(inv_freq=f, positions=pos.to(torch.int32).to(DEV), interleaved=inter) if rot else {}
    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    if Hq:
        kw.update(q=q, q_out=q_out)
    dash.kv_write(k, v, kc, vc, slots.to(DEV), k_scale=ks, v_scale=vs, **kw)
    no_error()
    x = qkv.double().numpy()
    turned = V.rope(x[:, :Hq + Hkv], pos.numpy()[:, None], f.numpy(), 1.0, inter) if rot else x[:, :Hq + Hkv]
    bound = rope_bound(x[:, :Hq + Hkv], f if rot else [], 1.0, inter, True, turned) if rot else 0 * turned
    if Hq:
        d = np.abs(q_out.double().cpu().numpy() - turned[:, :Hq])
        assert (d <= bound[:, :Hq])[np.isfinite(turned[:, :Hq])].all()
    keep = (slots >= 0).numpy()
    p, o = slots[keep] // page, slots[keep] % page
    touched = np.zeros((kc.shape[0], page), dtype=bool)
    touched[p, o] = True
    # values: never rotated, so every step is one fp32 operation: equal bits
    vw = qkv[keep][:, Hq + Hkv:]
    if quant:
        code, scale = quantised_nan(vw)
        assert torch.equal(vs.cpu()[p, :, o], scale)
        got = raw(vc).cpu()[p, :, o]
        nan = torch.isnan(vw)
        assert torch.equal(got[~nan], raw(code)[~nan]) and (got[nan] & 0x7f == 0x7f).all()
        kscale = ks.cpu().double().numpy()[p, :, o]
        kval = kc.cpu().float()[p, :, o].double().numpy() * kscale[..., None]
        ref = turned[keep][:, Hq:]
        top = np.abs(ref).max(-1) / 448.0
        assert (np.abs(kscale - top) <= 2.0 ** -18 * top + 2.0 ** -126).all()
        # half a step of e4m3: 2^-4 of the value, or 2^-10 scales among the smallest; fp32's errors before the rounding
        fp32 = rope_bound(x[keep][:, Hq:Hq + Hkv], f if rot else [], 1.0, inter, False, ref) if rot else 0 * ref
        lim = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * kscale[..., None]) * 1.0001 + 2 * fp32 + 2.0 ** -20 * np.abs(ref)
        assert (np.abs(kval - ref) <= lim).all()
    else:
        assert same_nan(vc.cpu()[p, :, o], vw)
        got = kc.cpu()[p, :, o].double().numpy()
        assert (np.abs(got - turned[keep][:, Hq:]) <= bound[keep][:, Hq:]).all()
    # cells of no token keep what they held
    mark = 3 if quant else 3.0
    for c in (kc, vc):
        rest = raw(c).cpu().permute(0, 2, 1, 3)[torch.from_numpy(~touched)]
        assert (rest == mark).all()
    if quant:
        assert (ks.cpu().permute(0, 2, 1)[torch.from_numpy(~touched)] == 9.0).all()


def quantised_nan(x):
    x = x.float()
    scale = (torch.nan_to_num(x, nan=0.0, posinf=float("inf")).abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)
    return (x / scale[..., None]).to(E4M3), scale


def same_nan(a, b):
    na, nb = torch.isnan(a), torch.isnan(b)
    return torch.equal(na, nb) and torch.equal(a[~na], b[~nb])


@pytest.mark.parametrize("quant", [False, True])
def test_write_reports_a_slot_past_the_cache(quant):
    case = (9, 2, 2, 64, 16, 64, False)
    qkv, slots, pos, (kc, vc), (ks, vs) = write_case(case, quant)
    before = [raw(t).clone() for t in (kc, vc)]
    slots[:] = kc.shape[0] * 16 + torch.arange(9) * 2 ** 33
    q, k, v = qkv.to(DEV).split([2, 2, 2], dim=1)
    dash.kv_write(k, v, kc, vc, slots.to(DEV), k_scale=ks, v_scale=vs)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info[0] == 1 and info[3] == kc.shape[0] * 16
    no_error()                                        # reported once
    assert torch.equal(before[0], raw(kc)) and torch.equal(before[1], raw(vc))


READS = [(1, 1, 1, 64, 16), (2, 2, 100, 128, 32), (3, 8, 300, 64, 64), (2, 3, 513, 128, 256), (5, 1, 130, 128, 128)]


@pytest.mark.parametrize("case", READS)
@pytest.mark.parametrize("quant", [False, True])
def test_read(case, quant):
    B, Hkv, S, D, page = case
    g = gen(8)
    lens = [int(x) for x in torch.randint(0, S + 1, (B,), generator=g)]
    lens[0] = S
    if B > 1:
        lens[1] = 0
    c = paged(g, lens, Hkv, D, page, quant)
    # outputs of another layout: tokens before heads
    k, v = (torch.full((B, S, Hkv, D), 77.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2) for _ in range(2))
    dash.kv_read(c.k_cache, c.v_cache, c.table, c.lens, k, v, **c.kw)
    no_error()
    for got, seqs, codes, scale in ((k, c.k, c.k_cache, c.k_scale), (v, c.v, c.v_cache, c.v_scale)):
        for b, n in enumerate(lens):
            # code * scale is exact in 64 bits here; one fp32 product, then one rounding to bf16
            ref = torch.from_numpy(seqs[b]).float().to(torch.bfloat16).transpose(0, 1)
            assert torch.equal(got[b, :, :n].cpu(), ref) and (got[b, :, n:] == 77.0).all()


def test_read_shorter_output_and_bad_pages():
    g = gen(9)
    c = paged(g, [60, 50, 40], 2, 64, 16, False)
    k, v = (torch.full((3, 2, 33, 64), 77.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dash.kv_read(c.k_cache, c.v_cache, c.table, c.lens, k, v)       # S < lens: the first S rows
    no_error()
    assert torch.equal(k[0].cpu().double(), torch.from_numpy(c.k[0][:33]).transpose(0, 1))
    table = c.table.clone()
    table[1, 1] = 10 ** 6
    lens = c.lens.clone()
    lens[2] = 10 ** 6
    v.fill_(77.0)
    dash.kv_read(c.k_cache, c.v_cache, table, lens, k, v)
    code, info = dash.get_status_paged()
    assert code == dash.ERR_PAGE and info[0] == 2 and info[1] in (1, 2)
    assert (v[1, :, 16:32] == 77.0).all() and torch.equal(v[1, :, :16].cpu().double(), torch.from_numpy(c.v[1][:16]).transpose(0, 1))
    assert torch.equal(v[0].cpu().double(), torch.from_numpy(c.v[0][:33]).transpose(0, 1))


def test_write_then_read_round_trip():
    T, Hkv, D, page = 77, 3, 128, 16
    x, y = randn(gen(10), T, Hkv, D), randn(gen(11), T, Hkv, D)
    N = 6
    table = torch.randperm(N, generator=gen(12))[:5].to(torch.int32)[None]
    j = torch.arange(T)
    slots = table[0].long()[j // page] * page + j % page
    for quant in (False, True):
        shape = (N, Hkv, page, D)
        kc, vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV).view(E4M3) if quant else
                  torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kw = dict(k_scale=torch.zeros(shape[:3], device=DEV), v_scale=torch.zeros(shape[:3], device=DEV)) if quant else {}
        dash.kv_write(x.to(DEV), y.to(DEV), kc, vc, slots.to(DEV), **kw)
        k, v = (torch.zeros(1, Hkv, T, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        dash.kv_read(kc, vc, table.to(DEV), torch.tensor([T], dtype=torch.int32, device=DEV), k, v, **kw)
        no_error()
        for got, src in ((k, x), (v, y)):
            if quant:
                code, scale = quantised(src)
                src = (code.float() * scale[..., None]).to(torch.bfloat16)
            assert torch.equal(got[0].transpose(0, 1).cpu(), src)
