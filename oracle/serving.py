"""Plain fp64 rotary positions, cache quantisation and attention over a paged
cache (numpy, one vector or row at a time where that is clearest).

Definitions: the rotation of value pairs by position * frequency and its
transpose; one scale per vector with e4m3 values (3 fraction bits, least
exponent -6, largest 448, nearest even); softmax attention of a sequence's
newest tokens over its cached keys with the diagonal at the sequence's end.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def rope(x, positions, inv_freq, factor=1.0, interleaved=False, inverse=False):
    """x [..., D]; positions broadcast to x.shape[:-1]; inv_freq [rot/2]."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    rot = 2 * f.size
    # positions are whole numbers: reduce the product modulo one turn in extended precision
    turns = np.asarray(positions, dtype=np.longdouble)[..., None] * (f.astype(np.longdouble) / (2 * np.pi))
    ang = ((turns - np.floor(turns)) * (2 * np.pi)).astype(np.float64)
    c, s = factor * np.cos(ang), factor * np.sin(ang)
    if inverse:
        s = -s
    y = x.copy()
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def rope_freqs(rot, base, scaling="none", scale=1.0, trained=0, lo=1.0, hi=4.0):
    """(frequencies, factor), written pair by pair."""
    if scaling == "base":
        base = base * scale ** (rot / (rot - 2))
    out, factor = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        turns = trained * f / (2 * math.pi)
        if scaling == "linear":
            f /= scale
        elif scaling == "wave":
            if turns < lo:
                f /= scale
            elif turns <= hi:
                t = (turns - lo) / (hi - lo)
                f = (1 - t) * f / scale + t * f
        elif scaling == "ramp":
            at = lambda n: rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), rot - 1)
            t = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
            f = f / scale * t + f * (1 - t)
            factor = 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
        out.append(f)
    return np.array(out), factor


def e4m3_round(x):
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)                       # |x| = m 2^e, m in [1/2, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def quantise(x):
    """(values on the e4m3 grid, scale) of vectors x [..., D]; code * scale stands for x."""
    x = np.asarray(x, dtype=np.float64)
    scale = np.maximum(np.abs(x).max(-1) / E4M3_MAX, 2.0 ** -126)
    return e4m3_round(x / scale[..., None]), scale


def attend(q, k, v, first, causal=True, window=0):
    """q [n, Hq, D] at positions first.., k, v [len, Hkv, D] -> o [n, Hq, D], lse [n, Hq]."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    pos = first + np.arange(n)
    j = np.arange(k.shape[0])
    seen = np.ones((n, j.size), dtype=bool)
    if causal:
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
    rows = seen.any(1)
    for h in range(Hq):
        x = (q[:, h] @ k[:, h // G].T) / math.sqrt(D)
        x[~seen] = -np.inf
        x = x[rows]
        m = x.max(1, initial=-np.inf, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(1, keepdims=True)
        o[rows, h] = (p / l) @ v[:, h // G]
        lse[rows, h] = (m + np.log(l))[:, 0]
    return o, lse


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise4(x, exp):
    """(values on the e2m1 grid, scale) of vectors x [..., D]: 16 values share an e4m3 scale in units of 2^exp;
    code * scale, the scale [..., D / 16] with its unit, stands for x."""
    b = np.asarray(x, dtype=np.float64)
    b = b.reshape(b.shape[:-1] + (-1, 16))
    s = e4m3_round(np.clip(np.abs(b).max(-1) / 6.0 * 2.0 ** -exp, 2.0 ** -9, E4M3_MAX)) * 2.0 ** exp
    y = np.minimum(np.abs(b) / s[..., None], 6.0)
    i = np.searchsorted(E2M1, y, side="left")            # E2M1[i - 1] < y <= E2M1[i]
    lo, hi = E2M1[np.maximum(i - 1, 0)], E2M1[i]
    mid = (lo + hi) / 2
    up = (y > mid) | ((y == mid) & (i % 2 == 0))         # ties to the even code
    return (np.where(up, hi, lo) * np.sign(b)).reshape(np.asarray(x).shape), s
