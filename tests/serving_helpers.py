"""Paged caches, references and bounds of the serving tests."""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import numpy as np
import torch

from oracle import serving as V
from tile_scheduling_persistent_gb300 import dash

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def randn(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def quantised(x):
    """x [..., D] on the CPU as (e4m3 codes, fp32 scale), in fp32 as documented."""
    x = x.float()
    scale = (x.abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)
    return (x / scale[..., None]).to(E4M3), scale


def raw(t):
    return t.view(torch.uint8) if t.dtype is E4M3 else t


@dataclass
class Paged:
    """B sequences' keys and values in shuffled pages; every cell that holds no token is NaN, every
    table entry behind the last page is out of range."""
    k: list           # per sequence [len, Hkv, D], fp64 values that the cache stands for
    v: list
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: torch.Tensor | None
    v_scale: torch.Tensor | None
    table: torch.Tensor
    lens: torch.Tensor
    kw: dict = field(default_factory=dict)


def paged(g, lens, Hkv, D, page, quant, extra_pages=2, sigma=1.0, max_len=None):
    lens = list(lens)
    width = max(-(-max(lens + [max_len or 0]) // page), 1)
    used = [-(-n // page) for n in lens]
    N = sum(used) + extra_pages
    order = torch.randperm(N, generator=g)
    shape = (N, Hkv, page, D)
    caches, scales, seqs = [], [], []
    tables = torch.full((len(lens), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        tables[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    for _ in range(2):
        c = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        s = torch.full(shape[:3], float("nan"))
        if quant:
            c = torch.full(shape, 0x7f, dtype=torch.uint8).view(E4M3)
        out = []
        for b, n in enumerate(lens):
            x = (torch.randn(n, Hkv, D, generator=g) * sigma).to(torch.bfloat16)
            j = torch.arange(n)
            p, o = tables[b].long()[j // page] if n else j, j % page
            if quant:
                q, sc = quantised(x)
                raw(c)[p, :, o] = raw(q)
                s[p, :, o] = sc
                out.append(q.float().double().numpy() * sc.double().numpy()[..., None])
            else:
                c[p, :, o] = x
                out.append(x.double().numpy())
        caches.append(c.to(DEV))
        scales.append(s.to(DEV) if quant else None)
        seqs.append(out)
    kw = dict(k_scale=scales[0], v_scale=scales[1]) if quant else {}
    return Paged(seqs[0], seqs[1], caches[0], caches[1], scales[0], scales[1], tables.to(DEV),
                 torch.tensor(lens, dtype=torch.int32, device=DEV), kw)


def run_attn(c: Paged, q, n, causal=True, window=None, pad=0, max_q=None, use_cu=True, want_lse=True, **kw):
    """o, lse of packed q (CPU or CUDA) whose sequences have n[b] new tokens; buffers start at a mark."""
    q = q.to(DEV)
    T, Hq, D = q.shape
    o = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 77.0, device=DEV) if want_lse else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV) if use_cu else None
    dash.attn_paged(q, c.k_cache, c.v_cache, c.table, c.lens, o, cu_q=cu, max_q=max(n) if max_q is None else max_q, lse=lse,
                    causal=causal, window=window, **c.kw, **kw)
    return o, lse


def check_attn(c: Paged, q, n, o, lse, causal=True, window=None):
    """Against the 64-bit oracle, element by element.  With A = sum_j P_j |v_j| the error of o is at most
      2^-8 A      each P_j is rounded to bf16 (half a step: 2^-8 relative) before the product with v
    + 2^-8 |o|    o itself is rounded to bf16
    + 2^-10 A     fp32: a score is a sum of D <= 128 products, off by at most 130 * 2^-23 * scale * sum|q k| (the sum's
                  absolute values stay below 12 * sqrt(D) for these inputs: 2e-4), which moves P by that much, and its
                  normalisation by as much again: 4e-4 < 2^-11; exponentials and sums add less than 2^-12.
    lse is off by the scores' error and fp32's: 2^-12 + 2^-20 |lse|."""
    o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy() if lse is not None else None
    at = 0
    for b, m in enumerate(n):
        ln = c.k[b].shape[0]
        ro, rl = V.attend(q[at:at + m].double().numpy(), c.k[b], c.v[b], ln - m, causal, window or 0)
        A, _ = V.attend(q[at:at + m].double().numpy(), c.k[b], np.abs(c.v[b]), ln - m, causal, window or 0)
        bound = (2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -8 * np.abs(ro)
        d = np.abs(o[at:at + m] - ro)
        assert (d <= bound).all(), "sequence %d: o off by %.3g of its bound" % (b, (d / np.maximum(bound, 1e-30)).max())
        if lse is not None:
            fin = np.isfinite(rl)
            got = lse[at:at + m]
            assert np.array_equal(np.isfinite(got), fin) and (got[~fin] == -np.inf).all()
            assert (np.abs(got[fin] - rl[fin]) <= 2.0 ** -12 + 2.0 ** -20 * np.abs(rl[fin])).all()
        at += m
    assert (o[at:] == 77.0).all() and (lse is None or (lse[at:] == 77.0).all()), "rows behind the last sequence changed"


def no_error():
    code, info = dash.get_status_paged()
    assert code == 0, (code, info)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16)) if a.dtype == torch.bfloat16 else torch.equal(
        a.view(torch.int32), b.view(torch.int32))


def rope_bound(x, inv_freq, factor, interleaved, bf16_out, ref):
    """|error| of a rotated value: the pair's absolute values times fp32's errors -- the angle's fraction of a turn is
    rounded to 24 bits (pi * 2^-24 rad), cos and sin are off by 2 units (2^-22), two products and a sum add 2^-22 --
    within 2^-20 together; then half a step of bf16: 2^-8 of the value, and 2^-134 below the least normal value 2^-126,
    where the steps are 2^-126 * 2^-7 = 2^-133 whatever the value (a relative bound has no room there)."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    rot = 2 * len(inv_freq)
    pair = x.copy()
    if interleaved:
        s = x[..., 0:rot:2] + x[..., 1:rot:2]
        pair[..., 0:rot:2] = pair[..., 1:rot:2] = s
    else:
        s = x[..., :rot // 2] + x[..., rot // 2:rot]
        pair[..., :rot // 2] = pair[..., rot // 2:rot] = s
    return pair * max(factor, 1.0) * 2.0 ** -20 + (2.0 ** -8 * 1.001 * np.abs(ref) + 2.0 ** -134 if bf16_out else 0.0)


def scale_of(D):
    return 1.0 / math.sqrt(D)
