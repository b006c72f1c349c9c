"""The serving and position operators as they are measured: cases, inputs, plain forms, the library's calls and 64-bit values.

Operators (the library computes attention over contiguous tensors; these are what a model puts around it):
  rope   rotary positions of queries and keys, forward, and backward (the inverse rotation of their gradients)
  write  new tokens' keys and values into a paged cache, rotated and quantised on the way
  read   a paged cache read back into contiguous tensors
  attn   attention of the newest tokens of each sequence over its paged cache

Layouts: q, o [T, Hq, D] packed tokens; k, v [T, Hkv, D]; training tensors [B, H, S, D]; cache pages
[num_pages, Hkv, page, D] in bf16, or e4m3 with one fp32 scale per token and head [num_pages, Hkv, page]; block tables
int32 [B, pages per sequence]; a slot is page * page_size + offset (negative: the token is not written).
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one training layer of the default workload: 32 query and 8 key heads of 16384 tokens, halves rotated
        dict(name="rope_train_16k", op="rope", B=1, Hq=32, Hkv=8, S=16384, D=128, rot=128, interleaved=False, scaling="none",
             inverse=False, x32=False, shared_pos=True, start=0),
        # its backward on the fp32 query gradient, half of the head rotated in neighbouring pairs, positions of a long context
        dict(name="rope_grad_partial", op="rope", B=4, Hq=16, Hkv=16, S=4096, D=128, rot=64, interleaved=True, scaling="ramp",
             inverse=True, x32=True, shared_pos=False, start=100000),
        # a decoding step of 64 sequences: one token each, rotated and quantised into its page
        dict(name="write_decode_64", op="write", T=64, Hq=32, Hkv=8, D=128, page=16, quant=True, rot=128, interleaved=False,
             scaling="wave", skip=False),
        # a ragged prompt written at once; padding tokens carry a negative slot
        dict(name="write_prompt_8k", op="write", T=8191, Hq=32, Hkv=8, D=128, page=64, quant=True, rot=128, interleaved=False,
             scaling="none", skip=True),
        # a short bf16 cache with 64-wide heads read back (a forked conversation)
        dict(name="read_short", op="read", B=2, Hkv=2, S=512, D=64, page=16, quant=False),
        # long quantised prefixes read back for a pass over contiguous tensors
        dict(name="read_prefix_16k", op="read", B=4, Hkv=8, S=16384, D=128, page=64, quant=True),
        # one chat: a single new token over about a thousand cached ones (latency)
        dict(name="attn_decode_one", op="attn", B=1, Hq=32, Hkv=8, D=128, page=16, quant=False, kv=1000, ragged=False, nq=1,
             chunks=0, causal=True, window=0, pad=0),
        # a serving batch: 64 sequences of ragged lengths up to 8192 over a quantised cache
        dict(name="attn_decode_batch", op="attn", B=64, Hq=32, Hkv=8, D=128, page=64, quant=True, kv=8192, ragged=True, nq=1,
             chunks=0, causal=True, window=0, pad=3),
        # very long contexts without shared heads
        dict(name="attn_decode_long", op="attn", B=2, Hq=16, Hkv=16, D=128, page=128, quant=False, kv=131071, ragged=False, nq=1,
             chunks=0, causal=True, window=0, pad=0),
        # several drafted tokens of each sequence checked at once
        dict(name="attn_verify_5", op="attn", B=16, Hq=32, Hkv=8, D=128, page=32, quant=False, kv=5000, ragged=True, nq=5,
             chunks=16, causal=True, window=0, pad=0),
        # a chunk of a long prompt over what is cached already
        dict(name="attn_chunk_4k", op="attn", B=1, Hq=32, Hkv=8, D=128, page=128, quant=False, kv=16384, ragged=False, nq=4096,
             chunks=1, causal=True, window=0, pad=0),
        # a mixed step: three prompts' chunks beside thirteen decoding sequences, sliding window, quantised, 64-wide heads
        dict(name="attn_mixed_window", op="attn", B=16, Hq=32, Hkv=8, D=64, page=16, quant=True, kv=8192, ragged=True, nq=700,
             chunks=3, causal=True, window=4096, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    hq, hkv = rng.choice([(32, 8), (16, 16), (32, 32), (16, 2), (28, 4), (8, 1), (6, 2)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    rot = rng.choice([d, d, d // 2])
    common = dict(rot=rot, interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "wave", "ramp"]))
    if op == "rope":
        b = rng.choice([1, 2, 4])
        inverse = rng.random() < 0.5
        return dict(op="rope", B=b, Hq=hq, Hkv=hkv, S=_log(rng, 1, 16384 // b), D=d, inverse=inverse,
                    x32=inverse and rng.random() < 0.5, shared_pos=rng.random() < 0.5, start=rng.choice([0, 5000, 900000]), **common)
    if op == "write":
        return dict(op="write", T=_log(rng, 1, 16000), Hq=hq, Hkv=hkv, D=d, page=page, quant=rng.random() < 0.6,
                    skip=rng.random() < 0.5, **common)
    if op == "read":
        b = _log(rng, 1, 64)
        return dict(op="read", B=b, Hkv=hkv, S=_log(rng, 1, 65536 // b), D=d, page=page, quant=rng.random() < 0.6)
    shape = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    base = dict(op="attn", Hq=hq, Hkv=hkv, D=d, page=page, quant=rng.random() < 0.5, ragged=rng.random() < 0.7,
                causal=rng.random() < 0.9, pad=rng.choice([0, 0, 1, 7]))
    if shape == "decode":
        b = _log(rng, 1, 128)
        kv, nq, chunks = _log(rng, 1, 131072 // b), 1, 0
    elif shape == "verify":
        b = _log(rng, 1, 32)
        kv, nq = _log(rng, 64, 65536 // b), rng.randint(2, 8)
        chunks = b
    elif shape == "chunk":
        b = rng.choice([1, 1, 2, 3])
        kv = _log(rng, 64, 16384 // b)
        nq, chunks = _log(rng, 1, min(kv, 4096)), b
    else:
        b = _log(rng, 4, 24)
        kv = _log(rng, 512, 8192)
        nq, chunks = _log(rng, 32, 512), rng.randint(1, 3)
    return dict(base, B=b, kv=kv, nq=nq, chunks=min(chunks, b), window=rng.choice([0, 0, _log(rng, 1, 8192)]) if base["causal"] else 0)


# --------------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int64)


def _inv_freq(rot, scaling):
    """Radians per position of each rotated pair, and the factor on the rotated values: a host table in 64 bits, as a
    model keeps it. linear: positions divided by 4. wave: pairs whose wavelength passes the trained length divided by
    8, with a smooth passage. ramp: a blend by the number of turns over the trained length, and the values' factor."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 500000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    turns = 8192.0 * f / (2.0 * math.pi)
    if scaling == "wave":
        t = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        return f * (t + (1.0 - t) / 8.0), 1.0
    if scaling == "ramp":
        lo, hi = (rot * math.log(8192.0 / (n * 2.0 * math.pi)) / (2.0 * math.log(500000.0)) for n in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        t = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (t + (1.0 - t) / 16.0), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _quantised(x):
    """x [..., D] as e4m3 codes and one fp32 scale for each vector."""
    x = x.float()
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    return (x / scale[..., None]).to(E4M3), scale


def _cache(g, c, pages, filled):
    shape = (pages, c["Hkv"], c["page"], c["D"])
    s = {}
    for n in ("k", "v"):
        x = _normal(g, *shape) if filled else torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        if c["quant"]:
            s[n + "_cache"], s[n + "_scale"] = _quantised(x)
        else:
            s[n + "_cache"], s[n + "_scale"] = x, None
    return s


def _tables(g, B, pages_each, extra=5):
    pages = B * pages_each + extra
    return pages, torch.randperm(pages, generator=g, device=DEV)[:B * pages_each].to(torch.int32).reshape(B, pages_each).contiguous()


def _attn_lens(c, g):
    """(kv lengths, new tokens) of each sequence: whole numbers from the case alone where not ragged."""
    B, kv, nq, chunks = c["B"], c["kv"], c["nq"], c["chunks"]
    n = torch.ones(B, dtype=torch.int64, device=DEV)
    n[:chunks] = nq
    if c["ragged"] and chunks < B:
        n[:chunks] = _ints(g, max(1, nq // 2), nq, chunks) if chunks else 1
        if chunks:
            n[0] = nq
    lens = _ints(g, 1, kv, B) if c["ragged"] else torch.full((B,), kv, dtype=torch.int64, device=DEV)
    lens[0] = kv
    lens = torch.maximum(lens, torch.minimum(n, torch.full_like(n, kv)))
    return lens, n


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "rope":
        first = torch.float32 if c["x32"] else torch.bfloat16
        s["q"] = _normal(g, c["B"], c["Hq"], c["S"], c["D"], dtype=first)
        s["k"] = _normal(g, c["B"], c["Hkv"], c["S"], c["D"])
        s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty_like(s["k"])
        at = torch.arange(c["S"], device=DEV, dtype=torch.int64)[None] + c["start"]
        if not c["shared_pos"]:  # packed documents: each row of the batch starts somewhere else
            at = at + _ints(g, 0, 1000, c["B"])[:, None]
        s["positions"] = (at[0] if c["shared_pos"] else at).to(torch.int32).contiguous()
        s["inv_freq"], s["factor"] = _inv_freq(c["rot"], c["scaling"])
    elif c["op"] == "write":
        T = c["T"]
        # queries, keys and values of one projection lie side by side in a row
        s["qkv"] = _normal(g, T, c["Hq"] + 2 * c["Hkv"], c["D"])
        s["q"], s["k"], s["v"] = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["q_out"] = torch.empty(T, c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
        pages = -(-T // c["page"]) + 3
        s.update(_cache(g, c, pages, filled=False))
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * c["page"] + torch.arange(c["page"], device=DEV)
        s["slots"] = slots.reshape(-1)[:T].to(torch.int64).contiguous()
        if c["skip"]:
            s["slots"][T - T // 16:] = -1
        s["positions"] = _ints(g, 0, 130000, T).to(torch.int32)
        s["inv_freq"], s["factor"] = _inv_freq(c["rot"], c["scaling"])
    else:
        S = c["S"] if c["op"] == "read" else c["kv"]
        pages, s["table"] = _tables(g, c["B"], -(-S // c["page"]))
        s.update(_cache(g, c, pages, filled=True))
        if c["op"] == "read":
            lens = _ints(g, max(1, S // 2), S, c["B"])
            lens[0] = S
            s["lens"] = lens.to(torch.int32)
            for n in ("k", "v"):
                s[n + "_out"] = torch.zeros(c["B"], c["Hkv"], S, c["D"], dtype=torch.bfloat16, device=DEV)
        else:
            lens, n = _attn_lens(c, g)
            cu = torch.zeros(c["B"] + 1, dtype=torch.int64, device=DEV)
            cu[1:] = n.cumsum(0)
            T = c["chunks"] * c["nq"] + c["B"] - c["chunks"] + c["pad"]  # the step's buffers: rows past cu[B] are padding
            s["q"] = _normal(g, T, c["Hq"], c["D"])
            s["o"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(T, c["Hq"], dtype=torch.float32, device=DEV)
            s["lens"], s["cu"] = lens.to(torch.int32), cu.to(torch.int32)
            s["max_q"] = int(n.max())
    return s


# ---------------------------------------------------------------------------------------------------------- plain forms
def _rotated(x, positions, inv_freq, factor, rot, interleaved, inverse=False):
    """x [..., D] in 32 bits with its first `rot` values rotated by positions (shape of x without the last axis, or
    broadcast to it). The angles are taken in 64 bits: far positions lose them in 32."""
    ang = positions.double()[..., None] * inv_freq.to(x.device)
    cos, sin = (ang.cos() * factor).float(), (ang.sin() * factor).float()
    sin = -sin if inverse else sin
    x, r = x.float(), x[..., :rot].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _plain_write(s):
    c = s["case"]
    at = s["positions"].long()[:, None]
    turn = (s["inv_freq"], s["factor"], c["rot"], c["interleaved"])
    s["q_out"].copy_(_rotated(s["q"], at, *turn))
    ok = s["slots"] >= 0
    slot = s["slots"][ok]
    page, off = slot // c["page"], slot % c["page"]
    for n, x in (("k", _rotated(s["k"], at, *turn)), ("v", s["v"].float())):
        x = x[ok]
        if c["quant"]:
            x, scale = _quantised(x)
            s[n + "_scale"][page, :, off] = scale
        _bytes_of(s[n + "_cache"])[page, :, off] = _bytes_of(x if c["quant"] else x.to(torch.bfloat16))


def _gathered(s, n):
    """The sequences' cached vectors [B, Hkv, pages * page, D] in 32 bits."""
    t = s["table"].long()
    x = _bytes_of(s[n + "_cache"])[t]
    x = x.view(E4M3).float() if s[n + "_scale"] is not None else x.float()
    if s[n + "_scale"] is not None:
        x = x * s[n + "_scale"][t][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_read(s):
    ok = (torch.arange(s["k_out"].shape[2], device=DEV) < s["lens"][:, None])[:, None, :, None]
    for n in ("k", "v"):
        out = s[n + "_out"]
        out.copy_(torch.where(ok, _gathered(s, n)[:, :, :out.shape[2]].to(torch.bfloat16), out))


def _plain_attn(s):
    c = s["case"]
    B, Hkv, G, D = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    lens, cu = s["lens"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=DEV)
    row = (cu[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = _gathered(s, "k"), _gathered(s, "v")
    j = torch.arange(k.shape[2], device=DEV)
    pos = (lens - n)[:, None] + i
    seen = (j < lens[:, None])[:, None, :].expand(B, i.numel(), j.numel())
    if c["causal"]:
        seen = seen & (j <= pos[..., None])
        if c["window"]:
            seen = seen & (j > pos[..., None] - c["window"])
    x = (q @ k.transpose(2, 3)).view(B, Hkv, G, i.numel(), j.numel()) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - m).exp()
    del x
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, Hkv, G, i.numel(), D) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + total.log())[..., 0]
    ok = i < n[:, None]
    s["o"][row[ok]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[ok].to(torch.bfloat16)
    s["lse"][row[ok]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[ok]


def run(state):
    s, c = state, state["case"]
    if own:
        from tile_scheduling_persistent_gb300 import dash
    if c["op"] == "rope":
        if own:
            dash.rope(s["q"], s["q_out"], s["inv_freq"], positions=s["positions"], x2=s["k"], y2=s["k_out"],
                      interleaved=c["interleaved"], factor=s["factor"], inverse=c["inverse"])
        else:
            at = s["positions"] if c["shared_pos"] else s["positions"][:, None]
            for n in ("q", "k"):
                s[n + "_out"].copy_(_rotated(s[n], at, s["inv_freq"], s["factor"], c["rot"], c["interleaved"], c["inverse"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "write":
        if own:
            dash.kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                          inv_freq=s["inv_freq"], positions=s["positions"], interleaved=c["interleaved"], factor=s["factor"],
                          q=s["q"], q_out=s["q_out"])
        else:
            _plain_write(s)
        return {n: s[n] for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}
    if c["op"] == "read":
        if own:
            dash.kv_read(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["k_out"], s["v_out"], k_scale=s["k_scale"],
                         v_scale=s["v_scale"])
        else:
            _plain_read(s)
        return {"k": s["k_out"], "v": s["v_out"]}
    if own:
        dash.attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["o"], cu_q=s["cu"], max_q=s["max_q"],
                        lse=s["lse"], causal=c["causal"], window=c["window"] or None, k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        _plain_attn(s)
    return {"o": s["o"], "lse": s["lse"]}


# ----------------------------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    D = c["D"]
    if c["op"] == "rope":
        n = c["B"] * c["S"] * D
        elems = n * (c["Hq"] + c["Hkv"])
        moved = n * (c["Hq"] * (6 if c["x32"] else 4) + c["Hkv"] * 4)
        return {"bytes": moved + 4 * c["S"] * (1 if c["shared_pos"] else c["B"]), "flops": 3 * elems * c["rot"] // D}
    if c["op"] == "write":
        T, kept = c["T"], c["T"] - (c["T"] // 16 if c["skip"] else 0)
        out = kept * 2 * c["Hkv"] * (D + 4 if c["quant"] else 2 * D)
        return {"bytes": T * c["Hq"] * D * 4 + kept * 2 * c["Hkv"] * D * 2 + out + 12 * T,
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"] + (3 * kept * 2 * c["Hkv"] * D if c["quant"] else 0)}
    cell = (D + 4) if c["quant"] else 2 * D
    if c["op"] == "read":  # lengths are uniform between half and the whole: their mean
        tokens = (c["S"] + (c["B"] - 1) * 0.75 * c["S"]) * 2 * c["Hkv"]
        return {"bytes": tokens * (cell + 2 * D), "flops": tokens * D if c["quant"] else 0}
    # mean lengths: the first sequence has the full one, ragged others half of it; chunks of ragged mixed steps three quarters
    B, kv = c["B"], c["kv"]
    half = 0.5 if c["ragged"] else 1.0
    nbytes = flops = 0.0
    for b in range(B):
        n = c["nq"] if b < c["chunks"] else 1
        if c["ragged"] and 0 < b < c["chunks"] < B:
            n = max(1.0, 0.75 * n)
        length = kv if b == 0 else max(half * kv, min(n, kv))
        seen = length - (min(n, length) - 1) / 2 if c["causal"] else length
        if c["window"]:
            seen, length = min(seen, c["window"]), min(length, c["window"] + n)
        nbytes += length * 2 * c["Hkv"] * cell + n * c["Hq"] * (4 * D + 4)
        flops += 4.0 * n * seen * c["Hq"] * D
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------- exact
def _turned64(x, pos, freq, factor, rot, pairs, sign):
    """Complex multiplication of the value pairs by factor * e^(sign i angle)."""
    x = x.double()
    z = x[..., :rot].unflatten(-1, (rot // 2, 2) if pairs else (2, rot // 2))
    z = torch.complex(z[..., 0], z[..., 1]) if pairs else torch.complex(z[..., 0, :], z[..., 1, :])
    a = torch.remainder(pos.double().unsqueeze(-1) * freq.to(DEV), 2.0 * math.pi)
    z = z * torch.polar(torch.full_like(a, factor), sign * a)
    out = x.clone()
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _nearest_e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even: 3 fraction bits, least exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        pos = s["positions"] if c["shared_pos"] else s["positions"].unsqueeze(1)
        sign = -1.0 if c["inverse"] else 1.0
        return {n: _turned64(s[n], pos, s["inv_freq"], s["factor"], c["rot"], c["interleaved"], sign) for n in ("q", "k")}
    if c["op"] == "write":
        pos = s["positions"].unsqueeze(1)
        turn = (pos, s["inv_freq"], s["factor"], c["rot"], c["interleaved"], 1.0)
        out = {"q_out": _turned64(s["q"], *turn)}
        where = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][where]
        for n, x in (("k", _turned64(s["k"], *turn)), ("v", s["v"].double())):
            x = x[where].transpose(0, 1)  # [Hkv, kept, D]
            cache = torch.zeros(c["Hkv"], s[n + "_cache"].shape[0] * c["page"], c["D"], dtype=torch.float64, device=DEV)
            if c["quant"]:
                top = x.abs().max(dim=-1).values / E4M3_MAX
                x = _nearest_e4m3(x / top.unsqueeze(-1))
                scale = s[n + "_scale"].double().transpose(0, 1).reshape(c["Hkv"], -1).clone()
                scale[:, slot] = top
                out[n + "_scale"] = scale.unflatten(1, (-1, c["page"])).transpose(0, 1).contiguous()
            cache[:, slot] = x
            out[n + "_cache"] = cache.unflatten(1, (-1, c["page"])).transpose(0, 1).contiguous()
        return out
    lens = s["lens"].tolist()

    def cached(n, b, h, length):
        pages = s["table"][b].long()
        x = s[n + "_cache"][:, h].double()[pages].flatten(0, 1)
        if c["quant"]:
            x = x * s[n + "_scale"][:, h].double()[pages].flatten().unsqueeze(1)
        return x[:length]

    if c["op"] == "read":
        out = {n: s[n + "_out"].double() for n in ("k", "v")}
        for b in range(c["B"]):
            for h in range(c["Hkv"]):
                for n in ("k", "v"):
                    out[n][b, h, :lens[b]] = cached(n, b, h, lens[b])
        return out
    if sum(lens) * c["Hkv"] * s["max_q"] > 2 ** 33:
        return None
    o, lse = s["o"].double(), s["lse"].double()
    cu, G = s["cu"].tolist(), c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        at = torch.arange(n, device=DEV) + (lens[b] - n)
        j = torch.arange(lens[b], device=DEV)
        off = torch.zeros(n, lens[b], dtype=torch.bool, device=DEV)
        if c["causal"]:
            off |= j[None, :] > at[:, None]
            if c["window"]:
                off |= at[:, None] - j[None, :] >= c["window"]
        for h in range(c["Hkv"]):
            k, v = cached("k", b, h, lens[b]), cached("v", b, h, lens[b])
            for g in range(h * G, h * G + G):
                x = torch.einsum("id,jd->ij", s["q"][cu[b]:cu[b + 1], g].double(), k) / math.sqrt(c["D"])
                x[off] = -math.inf
                t = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                w[t == -math.inf] = 0.0
                o[cu[b]:cu[b + 1], g], lse[cu[b]:cu[b + 1], g] = w @ v, t
    return {"o": o, "lse": lse}
