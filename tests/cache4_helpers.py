"""Paged caches of 4 bits, their plain forms and bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import serving as V

from serving_helpers import DEV, E4M3, Paged

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def quantised4(x, exp):
    """x [..., D] on the CPU as (bytes [..., D / 2], e4m3 scales [..., D / 16]), in fp32 as documented."""
    b = x.float().unflatten(-1, (-1, 16))
    unit = 2.0 ** exp
    top = b.abs().amax(-1)
    finite = torch.isfinite(b).all(-1)
    scale = (torch.where(finite, top, torch.zeros_like(top)) / (6.0 * unit)).clamp(2.0 ** -9, 448.0).to(E4M3)
    y = b / (scale.float() * unit)[..., None]
    a = y.abs()
    code = sum((a > t).int() for t in (0.25, 1.25, 2.5, 5.0)) + sum((a >= t).int() for t in (0.75, 1.75, 3.5))
    code = (code + 8 * torch.signbit(y).int()).flatten(-2).to(torch.uint8)
    raw = torch.where(finite, scale.view(torch.uint8), torch.full_like(scale.view(torch.uint8), 0x7f))
    return code[..., 0::2] | (code[..., 1::2] << 4), raw.view(E4M3)


def values4(codes, scale, exp):
    """What they stand for, in 64 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return (VALUES.double()[c].unflatten(-1, (-1, 16)) * scale.float().double()[..., None]).flatten(-2) * 2.0 ** exp


def paged4(g, lens, Hkv, D, page, extra_pages=2, sigma=1.0, max_len=None, exps=(-3, -2)):
    """B sequences' keys and values in shuffled pages; every cell that holds no token has a NaN scale, every table entry
    behind the last page is out of range."""
    lens = list(lens)
    width = max(-(-max(lens + [max_len or 0]) // page), 1)
    used = [-(-n // page) for n in lens]
    N = sum(used) + extra_pages
    order = torch.randperm(N, generator=g)
    tables = torch.full((len(lens), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        tables[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    caches, scales, seqs = [], [], []
    for exp in exps:
        c = torch.randint(0, 256, (N, Hkv, page, D // 2), generator=g, dtype=torch.uint8)
        s = torch.full((N, Hkv, page, D // 16), 0x7f, dtype=torch.uint8)
        out = []
        for b, n in enumerate(lens):
            x = (torch.randn(n, Hkv, D, generator=g) * sigma).to(torch.bfloat16)
            j = torch.arange(n)
            p, o = tables[b].long()[j // page] if n else j, j % page
            q, sc = quantised4(x, exp)
            c[p, :, o], s[p, :, o] = q, sc.view(torch.uint8)
            out.append(values4(q, sc, exp).numpy())
        caches.append(c.to(DEV))
        scales.append(s.view(E4M3).to(DEV))
        seqs.append(out)
    kw = dict(k_scale=scales[0], v_scale=scales[1], k_exp=exps[0], v_exp=exps[1])
    return Paged(seqs[0], seqs[1], caches[0], caches[1], scales[0], scales[1], tables.to(DEV),
                 torch.tensor(lens, dtype=torch.int32, device=DEV), kw)


def check_attn4(c: Paged, q, n, o, lse, causal=True, window=None):
    """Against the 64-bit oracle, element by element.  With A = sum_j P_j |v_j| the error of o is at most
      2^-11 A            each P_j is rounded to fp16 (half a step) before the product with v, which is exact in fp16
    + 2^-32 sum_j |v_j|  or, far below the row's largest, to 2^-32 of it (the largest P_j is at most 1)
    + 2^-8 |o|           o itself is rounded to bf16
    + 2^-10 A            fp32: a score is a sum of D <= 128 products, off by at most 130 * 2^-23 * scale * sum|q k| (the
                         sum's absolute values stay below 12 * sqrt(D) for these inputs: 2e-4), which moves P by that much,
                         and its normalisation by as much again: 4e-4 < 2^-11; exponentials and sums add less than 2^-12.
    lse is off by the scores' error and fp32's: 2^-12 + 2^-20 |lse|."""
    o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy() if lse is not None else None
    at = 0
    for b, m in enumerate(n):
        ln = c.k[b].shape[0]
        rows = q[at:at + m].double().numpy()
        ro, rl = V.attend(rows, c.k[b], c.v[b], ln - m, causal, window or 0)
        A, _ = V.attend(rows, c.k[b], np.abs(c.v[b]), ln - m, causal, window or 0)
        G = q.shape[1] // c.v[b].shape[1]
        total = np.repeat(np.abs(c.v[b]).sum(0), G, axis=0)[None] if ln else 0.0
        bound = (2.0 ** -11 + 2.0 ** -10) * A + 2.0 ** -32 * total + 2.0 ** -8 * np.abs(ro)
        d = np.abs(o[at:at + m] - ro)
        assert (d <= bound).all(), "sequence %d: o off by %.3g of its bound" % (b, (d / np.maximum(bound, 1e-30)).max())
        if lse is not None:
            fin = np.isfinite(rl)
            got = lse[at:at + m]
            assert np.array_equal(np.isfinite(got), fin) and (got[~fin] == -np.inf).all()
            assert (np.abs(got[fin] - rl[fin]) <= 2.0 ** -12 + 2.0 ** -20 * np.abs(rl[fin])).all()
        at += m
    assert (o[at:] == 77.0).all() and (lse is None or (lse[at:] == 77.0).all()), "rows behind the last sequence changed"
