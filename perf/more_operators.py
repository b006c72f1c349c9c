"""The operators of a paged cache held in 4 bits, and of its pages, as they are measured: cases, inputs, plain forms, the
library's calls and 64-bit values.

Operators:
  store    prompts' keys and values rotated and written into a cache of 4 bits, and the prefix read back for a pass over
           contiguous tensors
  attn     attention of the newest tokens of each sequence over a cache of 4 bits
  branch   a round of drafted branches: each sequence forked into several, pages taken for their new tokens, the partly
           filled pages that they share copied in every layer, and in the end the branches dropped and their pages freed
  compact  the pages in use moved to the front of the pool, with the tables and the cached cells

A cache of 4 bits holds e2m1 values, two to a byte (the first in the low half), with an e4m3 scale for every 16 values of
a vector: k and v [num_pages, Hkv, page, D / 2] bytes, scales [num_pages, Hkv, page, D / 16]; a value stands for
code * scale * 2^exp, exp a number of the cache. refs[p] counts the table entries that hold page p; 0 is a free page.
Pages are taken in ascending order, for the rows in order.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
K_EXP, V_EXP = -3, -2  # the keys' and the values' scales are in units of 2^-3 and 2^-2 here
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one short turn of a chat, 64-wide heads, a quarter of them rotated in neighbouring pairs (latency)
        dict(name="store_turn", op="store", B=1, Hq=16, Hkv=4, S=130, D=64, page=16, rot=16, interleaved=True, ragged=False),
        # a batch of long prompts of ragged lengths, whole heads rotated by halves
        dict(name="store_prompts_16k", op="store", B=4, Hq=32, Hkv=8, S=16383, D=128, page=64, rot=128, interleaved=False,
             ragged=True),
        # one chat: a single new token over about a thousand cached ones (latency)
        dict(name="attn_decode_one", op="attn", B=1, Hq=32, Hkv=8, D=128, page=16, kv=1000, ragged=False, nq=1, chunks=0,
             causal=True, window=0, pad=0),
        # a serving batch: 64 sequences of ragged lengths up to 8192
        dict(name="attn_decode_batch", op="attn", B=64, Hq=32, Hkv=8, D=128, page=64, kv=8192, ragged=True, nq=1, chunks=0,
             causal=True, window=0, pad=3),
        # very long contexts, 64-wide heads, a key head for every pair of query heads
        dict(name="attn_decode_long", op="attn", B=3, Hq=32, Hkv=16, D=64, page=128, kv=262143, ragged=False, nq=1, chunks=0,
             causal=True, window=0, pad=0),
        # several drafted tokens of each sequence checked at once
        dict(name="attn_verify_5", op="attn", B=16, Hq=32, Hkv=8, D=128, page=32, kv=5000, ragged=True, nq=5, chunks=16,
             causal=True, window=0, pad=0),
        # a chunk of a long prompt over what is cached already
        dict(name="attn_chunk_2k", op="attn", B=1, Hq=32, Hkv=8, D=128, page=128, kv=8192, ragged=False, nq=2048, chunks=1,
             causal=True, window=0, pad=0),
        # a mixed step: three prompts' chunks beside thirteen decoding sequences, sliding window, 64-wide heads
        dict(name="attn_mixed_window", op="attn", B=16, Hq=32, Hkv=8, D=64, page=16, kv=8192, ragged=True, nq=700, chunks=3,
             causal=True, window=4096, pad=5),
        # two continuations of one short chat, a small cache (latency)
        dict(name="branch_chat", op="branch", R=1, fork=2, kv=200, new=1, Hkv=2, D=64, page=16, layers=2, kind="bf16"),
        # a serving batch of 32 sequences, each with four branches of up to 6 tokens, in four layers
        dict(name="branch_batch", op="branch", R=32, fork=4, kv=4096, new=6, Hkv=8, D=128, page=64, layers=4, kind="bf16"),
        # a small pool after a few conversations have ended
        dict(name="compact_small", op="compact", R=6, kv=300, pages=160, Hkv=2, D=64, page=16, layers=1, kind="e2m1"),
        # a large one, less than half in use
        dict(name="compact_pool", op="compact", R=64, kv=4096, pages=5000, Hkv=8, D=128, page=64, layers=2, kind="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "attn", "branch", "compact"])
    hq, hkv = rng.choice([(32, 8), (16, 16), (32, 32), (16, 2), (28, 4), (8, 1), (6, 2)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        b = _log(rng, 1, 16)
        return dict(op="store", B=b, Hq=hq, Hkv=hkv, S=_log(rng, 1, 65536 * 40 // (hq + 2 * hkv) // b), D=d, page=page,
                    rot=rng.choice([d, d // 2, 48, 16]), interleaved=rng.random() < 0.5, ragged=rng.random() < 0.7)
    if op in ("branch", "compact"):
        kind = rng.choice(["bf16", "e4m3", "e2m1"])
        layers = rng.randint(1, 3)
        if op == "branch":
            r = _log(rng, 1, 48)
            return dict(op="branch", R=r, fork=rng.randint(1, 4), kv=_log(rng, 1, 65536 // r), new=_log(rng, 1, 40), Hkv=hkv, D=d,
                        page=page, layers=layers, kind=kind)
        r, kv = _log(rng, 1, 64), _log(rng, 16, 1000)
        used = r * -(-kv // page)
        return dict(op="compact", R=r, kv=kv, pages=used + _log(rng, 1, 2 * used + 50), Hkv=hkv, D=d, page=page, layers=layers, kind=kind)
    shape = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    base = dict(op="attn", Hq=hq, Hkv=hkv, D=d, page=page, ragged=rng.random() < 0.7, causal=rng.random() < 0.9,
                pad=rng.choice([0, 0, 1, 7]))
    if shape == "decode":
        b = _log(rng, 1, 128)
        kv, nq, chunks = _log(rng, 1, 131072 // b), 1, 0
    elif shape == "verify":
        b = _log(rng, 1, 32)
        kv, nq = _log(rng, 64, 65536 // b), rng.randint(2, 8)
        chunks = b
    elif shape == "chunk":
        b = rng.choice([1, 1, 2, 3])
        kv = _log(rng, 64, 7168 // b)
        nq, chunks = _log(rng, 1, min(kv, 2048)), b
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


def _quantised(x, exp):
    """x [..., D] as e2m1 codes, two to a byte, and an e4m3 scale for every 16 values."""
    x = x.float().unflatten(-1, (-1, 16))
    unit = 2.0 ** exp
    scale = (x.abs().amax(-1) / (6.0 * unit)).clamp(2.0 ** -9, 448.0).to(E4M3)
    y = x / (scale.float() * unit)[..., None]
    a = y.abs()
    # ties go to the even code
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte()
    code = (code + (a > 5.0).byte() + 8 * torch.signbit(y).byte()).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scale, exp):
    """What they stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=DEV)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    return (table[c].unflatten(-1, (-1, 16)) * (scale.float() * 2.0 ** exp)[..., None]).flatten(-2)


def _cells(g, c, pages, kind, filled):
    """k and v of a cache, and their scales."""
    head = (pages, c["Hkv"], c["page"])
    D = c["D"]
    s = {}
    for n, exp in (("k", K_EXP), ("v", V_EXP)):
        s[n + "_scale"] = None
        if kind == "e2m1":
            if filled:
                made = [_quantised(_normal(g, min(512, pages - at), *head[1:], D), exp) for at in range(0, pages, 512)]
                s[n], s[n + "_scale"] = (torch.cat([m[i] for m in made]) for i in (0, 1))
            else:
                s[n] = torch.zeros(*head, D // 2, dtype=torch.uint8, device=DEV)
                s[n + "_scale"] = torch.zeros(*head, D // 16, dtype=torch.uint8, device=DEV).view(E4M3)
        elif kind == "e4m3":
            x = _normal(g, *head, D)
            s[n + "_scale"] = x.abs().amax(-1).float() / 448.0
            s[n] = (x / s[n + "_scale"][..., None]).to(E4M3)
        else:
            s[n] = _normal(g, *head, D)
    return s


def _inv_freq(rot):
    """Radians per position of each rotated pair: a host table in 64 bits, as a model keeps it."""
    return 500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2.0 / rot)


def _attn_lens(c, g):
    """(kv lengths, new tokens) of each sequence."""
    B, kv, nq, chunks = c["B"], c["kv"], c["nq"], c["chunks"]
    n = torch.ones(B, dtype=torch.int64, device=DEV)
    n[:chunks] = nq
    if c["ragged"] and 0 < chunks < B:
        n[:chunks] = _ints(g, max(1, nq // 2), nq, chunks)
        n[0] = nq
    lens = _ints(g, 1, kv, B) if c["ragged"] else torch.full((B,), kv, dtype=torch.int64, device=DEV)
    lens[0] = kv
    return torch.maximum(lens, n.clamp_max(kv)), n


def _cumulative(n):
    return torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), n.cumsum(0))).to(torch.int32)


def _rows_of_pages(g, lens, page, width, pages):
    """A table [rows, width] over a shuffled pool, -1 behind each row's last page, and the pages' counts."""
    held = torch.arange(width, device=DEV) < ((lens + page - 1) // page)[:, None]
    at = torch.cumsum(held.flatten().long(), 0).view(held.shape) - 1
    table = torch.where(held, torch.randperm(pages, generator=g, device=DEV)[at.clamp_min(0)], -1)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[table[held]] = 1
    return table.to(torch.int32).contiguous(), refs


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    page = c["page"]
    if c["op"] == "store":
        B, S = c["B"], c["S"]
        lens = _ints(g, max(1, S // 2), S, B) if c["ragged"] else torch.full((B,), S, dtype=torch.int64, device=DEV)
        lens[0] = S
        width = -(-S // page)
        s["table"] = torch.randperm(B * width + 3, generator=g, device=DEV)[:B * width].to(torch.int32).view(B, width).contiguous()
        j = torch.arange(S, device=DEV)
        slots = s["table"].long()[:, j // page] * page + j % page
        real = (j < lens[:, None])
        # the prompts' rows padded to one length: padding is not written
        s["slots"] = torch.where(real, slots, -1).flatten().contiguous()
        s["positions"] = j.to(torch.int32).repeat(B)
        s["lens"] = lens.to(torch.int32)
        # queries, keys and values of one projection lie side by side in a row
        s["qkv"] = _normal(g, B * S, c["Hq"] + 2 * c["Hkv"], c["D"])
        s["q"], s["k_new"], s["v_new"] = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["q_out"] = torch.empty(B * S, c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
        s.update(_cells(g, c, B * width + 3, "e2m1", filled=False))
        s["k_out"], s["v_out"] = (torch.zeros(B, c["Hkv"], S, c["D"], dtype=torch.bfloat16, device=DEV) for _ in range(2))
        s["inv_freq"] = _inv_freq(c["rot"])
    elif c["op"] == "attn":
        width = -(-c["kv"] // page)
        pages = c["B"] * width + 5
        s["table"] = torch.randperm(pages, generator=g, device=DEV)[:c["B"] * width].to(torch.int32).view(c["B"], width).contiguous()
        s.update(_cells(g, c, pages, "e2m1", filled=True))
        lens, n = _attn_lens(c, g)
        T = c["chunks"] * c["nq"] + c["B"] - c["chunks"] + c["pad"]  # the step's buffers: rows past cu[B] are padding
        s["q"] = _normal(g, T, c["Hq"], c["D"])
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(T, c["Hq"], dtype=torch.float32, device=DEV)
        s["lens"], s["cu"], s["max_q"] = lens.to(torch.int32), _cumulative(n), int(n.max())
    else:
        R, kv = c["R"], c["kv"]
        lens = _ints(g, max(1, kv // 3), kv, R)
        lens[0] = kv
        if c["op"] == "branch":
            rows = R * (1 + c["fork"])
            width = -(-(kv + c["new"]) // page)
            pages = R * -(-kv // page) + R * c["fork"] * (-(-c["new"] // page) + 1) + 4
            at = torch.arange(R, device=DEV)
            s["parents"] = torch.cat((at, at.repeat_interleave(c["fork"]))).to(torch.int32)
            s["kept"] = torch.cat((at, torch.full((rows - R,), -1, device=DEV))).to(torch.int32)
            n = torch.cat((torch.zeros(R, dtype=torch.int64, device=DEV), _ints(g, 1, c["new"], rows - R)))
            n[R] = c["new"]
            s["cu"] = _cumulative(n)
            T = (rows - R) * c["new"]  # the step's buffers
            s["slots"] = torch.zeros(T, dtype=torch.int64, device=DEV)
            s["positions"] = torch.zeros(T, dtype=torch.int32, device=DEV)
            s["copies"] = torch.full((rows, 2), -1, dtype=torch.int32, device=DEV)
            for name in ("table1", "table2"):
                s[name] = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
            for name in ("lens1", "lens2"):
                s[name] = torch.zeros(rows, dtype=torch.int32, device=DEV)
        else:
            width, pages = -(-kv // page), c["pages"]
            s["copies"] = torch.full((pages // 2, 2), -1, dtype=torch.int32, device=DEV)
        s["table"], s["refs"] = _rows_of_pages(g, lens, page, width, pages)
        if c["op"] == "compact":
            s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["lens"] = lens.to(torch.int32)
        s["counts"] = torch.zeros(2, dtype=torch.int32, device=DEV)
        made = [_cells(g, c, pages, c["kind"], filled=True) for _ in range(c["layers"])]
        for n in ("k", "v", "k_scale", "v_scale"):
            s[n] = [m[n] for m in made if m[n] is not None]
    return s


# ---------------------------------------------------------------------------------------------------------- plain forms
def _rotated(x, positions, inv_freq, rot, interleaved):
    """x [..., D] in 32 bits with its first `rot` values rotated. The angles are taken in 64 bits."""
    ang = positions.double()[..., None] * inv_freq.to(x.device)
    cos, sin = ang.cos().float(), ang.sin().float()
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _gathered(s, n):
    """The sequences' cached vectors [B, Hkv, pages * page, D] in 32 bits."""
    t = s["table"].long()
    x = _values(s[n][t], _bytes_of(s[n + "_scale"])[t].view(E4M3), K_EXP if n == "k" else V_EXP)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_store(s):
    c = s["case"]
    at = s["positions"].long()[:, None]
    turn = (at, s["inv_freq"], c["rot"], c["interleaved"])
    s["q_out"].copy_(_rotated(s["q"], *turn))
    ok = s["slots"] >= 0
    slot = s["slots"][ok]
    where = (slot // c["page"], slice(None), slot % c["page"])
    for n, x, exp in (("k", _rotated(s["k_new"], *turn), K_EXP), ("v", s["v_new"], V_EXP)):
        codes, scale = _quantised(x[ok], exp)
        s[n][where] = codes
        _bytes_of(s[n + "_scale"])[where] = _bytes_of(scale)
    real = (torch.arange(c["S"], device=DEV) < s["lens"][:, None])[:, None, :, None]
    for n in ("k", "v"):
        out = s[n + "_out"]
        out.copy_(torch.where(real, _gathered(s, n)[:, :, :c["S"]].to(torch.bfloat16), out))


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


def _plain_fork(table, lens, parents, table_out, lens_out, refs, page):
    col = torch.arange(table.shape[1], device=DEV)
    from_row = parents.long().clamp_min(0)
    real = parents >= 0
    lens_out.copy_(torch.where(real, lens[from_row], 0))
    table_out.copy_(torch.where(col < ((lens_out + page - 1) // page)[:, None], table[from_row], -1))
    one = torch.ones((), dtype=torch.int32, device=DEV)
    refs.index_put_((table_out[table_out >= 0].long(),), one, accumulate=True)
    refs.index_put_((table[col < ((lens + page - 1) // page)[:, None]].long(),), -one, accumulate=True)


def _plain_extend(s, table, lens, refs, page):
    cu = s["cu"].long()
    R, n, old = lens.numel(), cu[1:] - cu[:-1], lens.long()
    row = torch.arange(R, device=DEV)
    held, want = (old + page - 1) // page, (old + n + page - 1) // page
    last = torch.where(held > 0, table[row, (held - 1).clamp_min(0)], 0).long()
    part = (n > 0) & (old % page != 0)  # rows that write into a page that they hold
    holders = torch.zeros(refs.numel(), dtype=torch.int64, device=DEV).index_add(0, last[part], torch.ones_like(last[part]))
    first = torch.full((refs.numel(),), R, dtype=torch.int64, device=DEV).scatter_reduce(0, last[part], row[part], "amin")
    copy = part & (refs[last] > 1) & ~((refs[last] == holders[last]) & (first[last] == row))
    need = want - held + copy
    taken = int(need.sum())
    pages = torch.nonzero(refs == 0)[:taken, 0]
    owner = row.repeat_interleave(need)
    k = torch.arange(taken, device=DEV) - (need.cumsum(0) - need)[owner]
    table[owner, held[owner] + k - copy[owner].long()] = pages.to(torch.int32)
    refs[pages] = 1
    refs.index_put_((last[copy],), torch.tensor(-1, dtype=torch.int32, device=DEV), accumulate=True)
    done = int(copy.sum())
    s["copies"][:done] = torch.stack((last[copy], table[row[copy], held[copy] - 1].long()), 1).to(torch.int32)
    s["counts"].copy_(torch.tensor([done, taken]))
    total = int(cu[-1])
    r = row.repeat_interleave(n)
    at = old[r] + torch.arange(total, device=DEV) - cu[r]
    s["positions"][:total], s["positions"][total:] = at.to(torch.int32), 0
    s["slots"][:total], s["slots"][total:] = table[r, at // page].long() * page + at % page, -1
    lens.add_(n.to(torch.int32))


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    at = torch.arange(refs.numel(), device=DEV)
    count = int(live.sum())
    src, dst = torch.nonzero(live & (at >= count))[:, 0], torch.nonzero(~live & (at < count))[:, 0]
    to = at.clone()
    to[src] = dst
    held = torch.arange(table.shape[1], device=DEV) < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    s["table_out"].copy_(torch.where(held, to[table.long().clamp_min(0)], table.long()))
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    s["copies"][:src.numel()] = torch.stack((src, dst), 1).to(torch.int32)
    s["counts"].copy_(torch.tensor([src.numel(), count]))


def _plain_copy(s):
    pair = s["copies"][:int(s["counts"][0])].long()
    for t in s["k"] + s["v"] + s["k_scale"] + s["v_scale"]:
        _bytes_of(t)[pair[:, 1]] = _bytes_of(t)[pair[:, 0]]


def _cells_of(s):
    """The cached cells as they were moved: nothing is computed with them."""
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


def run(state):
    s, c = state, state["case"]
    page = c["page"]
    if own:
        from tile_scheduling_persistent_gb300 import dash
    if c["op"] == "store":
        if own:
            scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_exp=K_EXP, v_exp=V_EXP)
            dash.kv_write(s["k_new"], s["v_new"], s["k"], s["v"], s["slots"], inv_freq=s["inv_freq"], positions=s["positions"],
                          interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"], **scales)
            dash.kv_read(s["k"], s["v"], s["table"], s["lens"], s["k_out"], s["v_out"], **scales)
        else:
            _plain_store(s)
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "attn":
        if own:
            dash.attn_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["o"], cu_q=s["cu"], max_q=s["max_q"], lse=s["lse"],
                            causal=c["causal"], window=c["window"] or None, k_scale=s["k_scale"], v_scale=s["v_scale"], k_exp=K_EXP,
                            v_exp=V_EXP)
        else:
            _plain_attn(s)
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "branch":
        if own:
            dash.pages_fork(s["table"], s["lens"], s["parents"], s["table1"], s["lens1"], s["refs"], page)
            dash.pages_extend(s["table1"], s["lens1"], s["refs"], page, s["slots"], s["positions"], s["copies"], s["counts"],
                              cu_new=s["cu"])
            dash.kv_copy(s["k"], s["v"], s["copies"], s["counts"], k_scales=s["k_scale"], v_scales=s["v_scale"])
            dash.pages_fork(s["table1"], s["lens1"], s["kept"], s["table2"], s["lens2"], s["refs"], page)
        else:
            _plain_fork(s["table"], s["lens"], s["parents"], s["table1"], s["lens1"], s["refs"], page)
            _plain_extend(s, s["table1"], s["lens1"], s["refs"], page)
            _plain_copy(s)
            _plain_fork(s["table1"], s["lens1"], s["kept"], s["table2"], s["lens2"], s["refs"], page)
        names = ("table1", "lens1", "table2", "lens2", "refs", "slots", "positions", "copies", "counts")
    else:
        if own:
            dash.pages_compact(s["table"], s["lens"], s["refs"], page, s["copies"], s["counts"], table_out=s["table_out"],
                               refs_out=s["refs_out"])
            dash.kv_copy(s["k"], s["v"], s["copies"], s["counts"], k_scales=s["k_scale"], v_scales=s["v_scale"])
        else:
            _plain_compact(s)
            _plain_copy(s)
        names = ("table_out", "refs_out", "copies", "counts")
    return dict({n: s[n] for n in names}, cells=_cells_of(s))


# ----------------------------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    D, page = c["D"], c["page"]
    cell4 = D // 2 + D // 16
    if c["op"] == "store":
        share = 0.75 if c["ragged"] else 1.0  # lengths are uniform between half and the whole: their mean
        rows, kept = c["B"] * c["S"], c["S"] + (c["B"] - 1) * share * c["S"]
        nbytes = rows * c["Hq"] * D * 4 + 12 * rows + kept * 2 * c["Hkv"] * (2 * D + cell4 + cell4 + 2 * D)
        return {"bytes": nbytes, "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"] + 4 * kept * 2 * c["Hkv"] * D}
    if c["op"] != "attn":
        cells = page * c["Hkv"] * {"bf16": 2 * D, "e4m3": D + 4, "e2m1": cell4}[c["kind"]] * 2 * c["layers"]  # of a page
        R, entries = c["R"], c["R"] * (0.67 * c["kv"] / page + 1)
        if c["op"] == "branch":  # nearly every branch shares a partly filled page with its sequence
            shared = R * c["fork"] * (page - 1) / page
            tables = entries * 4 * (2 + 3 * c["fork"]) + 12 * R * c["fork"] * c["new"] * 0.5
            return {"bytes": shared * 2 * cells + tables, "flops": 0}
        used = min(entries, c["pages"])
        moved = used * (1 - used / c["pages"])
        return {"bytes": moved * 2 * cells + 8 * entries + 8 * c["pages"], "flops": 0}
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
        nbytes += length * 2 * c["Hkv"] * cell4 + n * c["Hq"] * (4 * D + 4)
        flops += 4.0 * n * seen * c["Hq"] * D
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------- exact
def _turned64(x, pos, freq, rot, pairs):
    """Complex multiplication of the value pairs by e^(i angle)."""
    x = x.double()
    z = x[..., :rot].unflatten(-1, (rot // 2, 2) if pairs else (2, rot // 2))
    z = torch.complex(z[..., 0], z[..., 1]) if pairs else torch.complex(z[..., 0, :], z[..., 1, :])
    a = torch.remainder(pos.double().unsqueeze(-1) * freq.to(DEV), 2.0 * math.pi)
    z = z * torch.polar(torch.ones_like(a), a)
    out = x.clone()
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _nearest(x, fraction, least, most):
    """x (64 bits, not negative) on the grid of values with so many fraction bits and that least exponent, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -40))).clamp_min(least) - fraction)
    return (torch.round(x / step) * step).clamp_max(most)


def _held64(x, exp):
    """What a cache of 4 bits holds of x [..., D]."""
    b = x.unflatten(-1, (x.shape[-1] // 16, 16))
    scale = _nearest((b.abs().max(dim=-1).values / 6.0 * 2.0 ** -exp).clamp_min(2.0 ** -9), 3, -6, 448.0) * 2.0 ** exp
    y = b / scale.unsqueeze(-1)
    return (_nearest(y.abs(), 1, 0, 6.0) * torch.sign(y) * scale.unsqueeze(-1)).flatten(-2)


def _cached64(s, n, b, h, length):
    """The first `length` vectors of head h of sequence b, code by code."""
    pages = s["table"][b].long()
    raw = s[n][:, h][pages].flatten(0, 1)[:length].long()
    code = torch.empty(length, 2 * raw.shape[1], dtype=torch.int64, device=DEV)
    code[:, 0::2], code[:, 1::2] = raw % 16, raw // 16
    low, high = code % 2, (code // 2) % 4
    value = torch.where(high == 0, 0.5 * low.double(), (1.0 + 0.5 * low.double()) * torch.exp2(high.double() - 1.0))
    scale = s[n + "_scale"].view(torch.uint8)[:, h][pages].view(E4M3).flatten(0, 1)[:length].double()
    return value * torch.where(code >= 8, -1.0, 1.0) * scale.repeat_interleave(16, 1) * 2.0 ** (K_EXP if n == "k" else V_EXP)


def exact(case, seed):
    c = case
    if c["op"] in ("branch", "compact"):  # whole numbers and cells that are moved
        return None
    s = prepare(case, seed)
    if c["op"] == "store":
        turn = (s["positions"].unsqueeze(1), s["inv_freq"], c["rot"], c["interleaved"])
        out = {"q": _turned64(s["q"], *turn)}
        real = torch.arange(c["S"], device=DEV).unsqueeze(0) < s["lens"].unsqueeze(1)
        for n, x, exp in (("k", _turned64(s["k_new"], *turn), K_EXP), ("v", s["v_new"].double(), V_EXP)):
            held = _held64(x, exp).unflatten(0, (c["B"], c["S"])).transpose(1, 2)
            out[n] = held * real[:, None, :, None]
        return out
    lens = s["lens"].tolist()
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
            k, v = _cached64(s, "k", b, h, lens[b]), _cached64(s, "v", b, h, lens[b])
            for g in range(h * G, h * G + G):
                x = torch.einsum("id,jd->ij", s["q"][cu[b]:cu[b + 1], g].double(), k) / math.sqrt(c["D"])
                x[off] = -math.inf
                t = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                w[t == -math.inf] = 0.0
                o[cu[b]:cu[b + 1], g], lse[cu[b]:cu[b + 1], g] = w @ v, t
    return {"o": o, "lse": lse}
