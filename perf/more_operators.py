"""The serving operators around a paged cache held in 4 bits, as cases to be measured.

Four operators of a serving loop, in the order in which a program calls them:
rotation tables, plain and scaled for long contexts (`rope_table`); pages
handed out and taken back by the sequences' lengths, with the offsets,
positions and slots of the new tokens (`page_plan`); new tokens normalised,
rotated, quantised and appended to pages of 4-bit codes, and read back
(`append4`); attention of the new tokens over those pages, with a prefix that
the batch shares (`attend4`).

`run` computes them in plain torch where `own` is false and calls the
package's entry points where it is true.

The pages.  A page of one KV head is page_size / 16 blocks of 2560 bytes, each
16 tokens: 1024 bytes of key codes, 256 of key scales and zeros, the same for
the values.  Every 32 channels of a token have an fp16 scale s and zero z, and
a code c in 0..15 stands for z + s c.
  key codes     [token][c 4][group 4] words of 8 codes, channels 8 c .. 8 c + 7
                of the group: the even ones in the word's nibbles 0..3, the odd
                ones in 4..7
  key scales    [token][s, z][group] fp16
  value codes   [half 2][g 8][c 4][m 4] words, of channels 64 half + 16 m + g
                (low nibble) and + 8 (high nibble): byte b holds the token
                2 c + (b >> 1) + 8 (b & 1)
  value scales  [s, z][c 4][8s 2][group 4][odd 2] fp16, of token 8 8s + 2 c + odd
"""
import math

import numpy as np
import torch

own = False

D = 128                     # head dimension of the framework
G = 32                      # channels of a scale
BLOCK = 2560                # bytes of 16 tokens' keys and values
EPS = 1e-6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the rotation table of a short context, half of a head's channels: the smallest call, latency counts
        dict(name="rope_short", op="rope_table", positions=2048, start=0, rope=64, kind="plain", base=10000.0, factor=1.0,
             original=2048),
        # the table of a 131072-token context from a model trained on 8192, scaled by parts
        dict(name="rope_long", op="rope_table", positions=131072, start=0, rope=128, kind="parts", base=500000.0, factor=16.0,
             original=8192),
        # 16 sequences bring one sampled and four drafted tokens each, then roll back: some cross a page's border
        dict(name="pages_step", op="page_plan", batch=16, new=5, ragged=False, length=4096, page=64),
        # prompt chunks of up to 256 tokens of 512 sequences: many pages, many rows
        dict(name="pages_chunks", op="page_plan", batch=512, new=256, ragged=True, length=2048, page=16),
        # one decode step's tokens into pages of 64
        dict(name="append4_step", op="append4", dtype="bf16", batch=16, new=1, ragged=False, length=4096, page=64,
             hq=28, hkv=4, rope=128, interleaved=False, norm=True),
        # prompt chunks of different lengths in one batch, interleaved pairs on half of the channels, no norm
        dict(name="append4_chunks", op="append4", dtype="fp16", batch=32, new=611, ragged=True, length=1500, page=16,
             hq=24, hkv=8, rope=64, interleaved=True, norm=False),
        # a single sequence's decode step: latency
        dict(name="attend4_one", op="attend4", dtype="fp16", batch=1, new=1, ragged=False, shared=0, own=513, page=16,
             hq=24, hkv=8),
        # 16 sequences of up to 32768 tokens, nothing shared: the cache read at memory speed
        dict(name="attend4_long", op="attend4", dtype="bf16", batch=16, new=1, ragged=False, shared=0, own=32768, page=64,
             hq=28, hkv=4),
        # 64 sequences of up to 8191 tokens with as many KV heads as query heads: one row a KV head
        dict(name="attend4_heads", op="attend4", dtype="fp16", batch=64, new=1, ragged=False, shared=0, own=8191, page=32,
             hq=16, hkv=16),
        # decode of 32 sequences behind one 8192-token prompt
        dict(name="attend4_shared", op="attend4", dtype="fp16", batch=32, new=1, ragged=False, shared=8192, own=777,
             page=32, hq=24, hkv=8),
        # up to 5 tokens (one sampled, four drafted) of 32 sequences over 8192 tokens each
        dict(name="attend4_drafts", op="attend4", dtype="bf16", batch=32, new=5, ragged=True, shared=0, own=8192,
             page=64, hq=28, hkv=4),
        # prompt chunks of up to 512 tokens over a cache of 8192
        dict(name="attend4_chunks", op="attend4", dtype="bf16", batch=4, new=512, ragged=True, shared=0, own=8192, page=128,
             hq=24, hkv=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((24, 8), (28, 4), (32, 8), (16, 16), (8, 1), (5, 1), (12, 4))


def draw(rng):
    op = rng.choice(("rope_table", "page_plan", "append4", "append4", "attend4", "attend4", "attend4"))
    if op == "rope_table":
        kind = rng.choice(("plain", "linear", "ntk", "parts"))
        return dict(op=op, positions=_log(rng, 1, 131072), start=rng.choice((0, 0, _log(rng, 1, 1000000))),
                    rope=16 * rng.randint(1, 8), kind=kind, base=rng.choice((10000.0, 500000.0, 1000000.0)),
                    factor=1.0 if kind == "plain" else round(rng.uniform(1.5, 32.0), 2), original=rng.choice((2048, 4096, 8192)))
    page = rng.choice((16, 32, 64, 128))
    if op == "page_plan":
        batch = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, 65536 // batch))
        return dict(op=op, batch=batch, new=new, ragged=rng.random() < 0.5,
                    length=_log(rng, 1, max(2, min(32768, 1000000 // batch))), page=page)
    hq, hkv = rng.choice(HEADS)
    dtype = rng.choice(("fp16", "bf16"))
    batch = _log(rng, 1, 64)
    if op == "append4":
        new = _log(rng, 1, max(1, 16384 // batch))
        return dict(op=op, dtype=dtype, batch=batch, new=new, ragged=rng.random() < 0.5,
                    length=new + _log(rng, 1, max(2, 65536 // batch)), page=page, hq=hq, hkv=hkv,
                    rope=rng.choice((32, 48, 64, 128)), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6)
    new = rng.choice((1, 1, 2, 3, 5, 8, 17, 64))
    new = min(new, max(1, 512 // batch))
    shared = rng.choice((0, 1, 1)) * (_log(rng, 128, 32768) // page) * page
    most = max(64, min(32768, (1600000 if new <= 8 else 400000) // (batch * hkv)))
    return dict(op=op, dtype=dtype, batch=batch, new=new, ragged=rng.random() < 0.5, shared=shared,
                own=new + _log(rng, 1, most), page=page, hq=hq, hkv=hkv)


# ------------------------------------------------------------------ sizes that follow from a case

def _new_tokens(case):
    """Tokens that each sequence brings: `new`, or 1..new, spread, where the case is ragged."""
    b, n = case["batch"], case["new"]
    return [1 + (n - 1 - (i * 7919) % n) if case["ragged"] else n for i in range(b)]


def _own_lengths(case, most, new):
    """Tokens of each sequence (behind what is shared): from `most` down to about half of it."""
    b = case["batch"]
    return [max(n, most - i * most // (2 * b)) for i, n in zip(range(b), new)]


def _lengths(case):
    new = _new_tokens(case)
    if case["op"] == "attend4":
        return new, [case["shared"] + x for x in _own_lengths(case, case["own"], new)]
    return new, _own_lengths(case, case["length"], new)


def work(case):
    op = case["op"]
    if op == "rope_table":
        n = case["positions"] * case["rope"]
        return {"bytes": 4 * n, "flops": 20 * n}
    new, lengths = _lengths(case)
    n, b = sum(new), case["batch"]
    if op == "page_plan":
        # twice the lengths, counts and pages held, in and out, the offsets; the pages that change hands, both ways; a new
        # row's position and slot
        page = case["page"]
        taken = sum(-(-(x + k) // page) - -(-x // page) for k, x in zip(new, lengths))
        return {"bytes": 2 * (b * (4 + 16 + 8) + 4 * (b + 1)) + taken * 16 + n * 16, "flops": n}
    hq, hkv = case["hq"], case["hkv"]
    if op == "append4":
        # queries in and out, keys and values in, the new tokens' codes out, in again and their values out
        return {"bytes": n * ((2 * hq + 4 * hkv) * D * 2 + 2 * hkv * 160 + 4 * case["rope"]), "flops": n * (hq + 4 * hkv) * D * 8}
    shared = case["shared"]
    keys = shared + sum(x - shared for x in lengths)
    # query t of a sequence sees the tokens up to its own
    pairs = sum(t * x - t * (t - 1) // 2 for t, x in zip(new, lengths))
    return {"bytes": keys * hkv * 160 + n * hq * 2 * D * 2, "flops": pairs * hq * 4 * D}


# ------------------------------------------------------------------ the pages' layout

def _nibbles(x):
    return torch.stack([x & 15, x >> 4], -1)


def _bytes(x):
    return x[..., 0] | x[..., 1] << 4


def _fields(pages):
    """Views of pages [..., bytes]: key codes, key scales and zeros, value codes, value scales and zeros of each block."""
    x = pages.unflatten(-1, (-1, BLOCK))
    return (x[..., :1024].unflatten(-1, (16, 4, 4, 4)), x[..., 1024:1280].view(torch.float16).unflatten(-1, (16, 2, 4)),
            x[..., 1280:2304].unflatten(-1, (2, 8, 4, 4, 4)),
            x[..., 2304:].view(torch.float16).unflatten(-1, (2, 4, 2, 4, 2)))


def _move(x, n, order):
    """The last n dimensions in another order."""
    lead = x.dim() - n
    return x.permute(*range(lead), *[lead + i for i in order])


def _key_values(codes, sz):
    """[..., tokens, 128] fp32 of key codes [..., token, c, group, byte] and their scales."""
    x = _nibbles(codes).unflatten(-2, (2, 2))                      # token c group odd i nibble
    x = _move(x, 5, (1, 0, 3, 4, 2)).flatten(-4)                   # token group (c i nibble odd)
    return (x.float() * sz[..., 0, :, None].float() + sz[..., 1, :, None].float()).flatten(-2)


def _value_values(codes, sz):
    """[..., 16, 128] fp32 of value codes [..., half, g, c, m, byte] and their scales."""
    x = _nibbles(codes).unflatten(-2, (2, 2))                      # half g c m odd eight nibble
    x = _move(x, 7, (5, 2, 4, 0, 3, 6, 1)).flatten(-7, -5).flatten(-4)      # token channel
    s, z = (_move(t, 4, (1, 0, 3, 2)).flatten(-4, -2) for t in sz.unbind(-5))   # token group
    return (x.unflatten(-1, (4, G)).float() * s[..., None].float() + z[..., None].float()).flatten(-2)


def _quantise(x):
    """Codes, scales and zeros of rows [..., 128] (fp32 of the cache's type)."""
    x = x.unflatten(-1, (4, G))
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = ((hi - lo) / 15).clamp(max=65504).half(), lo.clamp(-65504, 65504).half()
    step = s.float()[..., None]
    c = torch.where(step > 0, torch.round((x - z.float()[..., None]) / torch.where(step > 0, step, 1.0)), 0.0)
    return c.clamp(0, 15).to(torch.uint8).flatten(-2), s, z


def _key_codes(c):
    """[..., 128] codes of a token -> its bytes [..., c, group, 4]."""
    x = c.unflatten(-1, (4, 4, 2, 2, 2))                           # group c i nibble odd
    return _bytes(_move(x, 5, (1, 0, 4, 2, 3))).flatten(-2)


def _value_codes(c):
    """[..., 128] codes of a token -> its bytes [..., half, m, g]."""
    return _bytes(_move(c.unflatten(-1, (2, 4, 2, 8)), 4, (0, 1, 3, 2)))


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """Angles a position of the rope / 2 pairs, and the factor of the cosines and sines, in 64 bits on the host."""
    d, base, factor = case["rope"], case["base"], case["factor"]
    if case["kind"] == "ntk":
        base = base * factor ** (d / (d - 2))
    f = base ** (-np.arange(0, d, 2, dtype=np.float64) / d)
    if case["kind"] == "linear":
        return f / factor, 1.0
    if case["kind"] != "parts":
        return f, 1.0
    # pairs with few turns in the context of the training are stretched, those with many stay, a line between
    turns = case["original"] * f / (2 * math.pi)
    stay = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * (stay + (1 - stay) / factor), 0.1 * math.log(factor) + 1.0


def _pairs_state(case, g, dev, n_positions):
    """The rotation table (cosines, then sines, of the rope/2 angles of a position) and the norm's weights."""
    half = case["rope"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    ang = torch.arange(n_positions, device=dev, dtype=torch.float64)[:, None] * freq
    s = {"cos_sin": torch.cat([ang.cos(), ang.sin()], 1).float(), "q_weight": None, "k_weight": None}
    if case["norm"]:
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(DTYPES[case["dtype"]])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    op = case["op"]
    if op == "rope_table":
        # a program makes one table a model: its base is what differs between them
        base = case["base"] * (1 + 1e-3 * float(torch.rand((), generator=g, device=dev)))
        return {"op": op, "case": dict(case, base=base)}
    new, lengths = _lengths(case)
    if op == "page_plan":
        return _prepare_plan(case, g, dev, new, lengths)
    dt, hq, hkv = DTYPES[case["dtype"]], case["hq"], case["hkv"]
    b, page, n = case["batch"], case["page"], sum(new)
    shared_pages = case.get("shared", 0) // page
    own_pages = -(-(max(lengths) - shared_pages * page) // page)
    n_pages = shared_pages + b * own_pages + 3
    # page ids in no order, as an allocator hands them out after a while
    ids = torch.randperm(n_pages, generator=g, device=dev)[:shared_pages + b * own_pages].to(torch.int32)
    table = torch.cat([ids[:shared_pages].expand(b, -1), ids[shared_pages:].view(b, own_pages)], 1).contiguous()
    pages = torch.empty(n_pages, hkv, page // 16 * BLOCK, dtype=torch.uint8, device=dev)
    s = {"op": op, "case": case, "table": table, "shared_pages": shared_pages, "pages": pages,
         "lengths": torch.tensor(lengths, dtype=torch.int64, device=dev),
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev), "max_new": max(new)}
    mean = 0.5 * torch.randn(2, hkv, 1, 1, D, generator=g, device=dev)    # keys and values have a mean a channel
    piece = max(1, (1 << 19) // (hkv * page))
    for i in range(0, n_pages, piece):                                    # in pieces: the fp32 normals are 13 times as large
        kc, ks, vc, vs = _fields(pages[i:i + piece])
        for t, (codes, sz) in enumerate(((kc, ks), (vc, vs))):
            x = torch.randn(*codes.shape[:3], 16, D, generator=g, device=dev) + mean[t]
            c, sc, z = _quantise(x.to(dt).float())
            if t == 0:
                codes.copy_(_key_codes(c))
                sz.copy_(torch.stack([sc, z], -2))
            else:                                                         # token = 8 eight + 2 c + odd
                y = _value_codes(c).unflatten(-4, (2, 4, 2))              # eight c odd half m g
                codes.copy_(_move(y, 6, (3, 5, 1, 4, 2, 0)).flatten(-2))
                sz.copy_(_move(torch.stack([sc, z], -3).unflatten(-2, (2, 4, 2)), 5, (0, 2, 1, 4, 3)))
    if op == "append4":
        qkv = torch.randn(n, hq + 2 * hkv, D, generator=g, device=dev).to(dt)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        s.update(_pairs_state(case, g, dev, max(lengths)))
    else:
        s["q"] = torch.randn(n, hq, D, generator=g, device=dev).to(dt)
    if own:  # the handle on the pages, and the attention's workspace, as a program keeps them
        from rank_latent_kv_gb300 import palu as P
        s["cache"] = P.PagedCache4(pages, table, s["lengths"], page, dt)
        if op == "attend4":
            s["workspace"] = s["cache"].attend_workspace(n, hq, s["max_new"], shared_pages)
    return s


def _prepare_plan(case, g, dev, new, lengths):
    b, page, n = case["batch"], case["page"], sum(new)
    held = [-(-x // page) for x in lengths]
    width = -(-max(x + k for x, k in zip(lengths, new)) // page) + 1
    n_pages = sum(-(-(x + k) // page) for x, k in zip(lengths, new)) + 7
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=dev)
    held_t = torch.tensor(held, **i32)
    col = torch.arange(width, device=dev)
    first = torch.cumsum(held_t.long(), 0) - held_t
    table = torch.where(col < held_t[:, None], ids[(first[:, None] + col).clamp(max=n_pages - 1)], 0).to(torch.int32)
    free = torch.zeros(n_pages, **i32)
    free[:n_pages - sum(held)] = ids[sum(held):]
    # the order of the sequences in the batch, so that other seeds have other lengths
    order = torch.randperm(b, generator=g, device=dev)
    len_t = torch.tensor(lengths, dtype=torch.int64, device=dev)[order].contiguous()
    s = {"op": "page_plan", "case": case, "table": table[order].contiguous(), "lengths": len_t, "before": len_t.clone(),
         "held": held_t[order].contiguous(), "free": free, "n_free": torch.tensor([n_pages - sum(held)], **i32),
         "new": torch.tensor(new, **i32)[order].contiguous(), "none": torch.zeros(b, **i32), "rows": n}
    if own:
        from rank_latent_kv_gb300 import palu as P
        s["pool"] = P.PagePool(s["table"], s["lengths"], page, held=s["held"], free_pages=free, n_free=s["n_free"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"rope_table": _rope_table, "page_plan": _page_plan, "append4": _append4, "attend4": _attend4}[s["op"]](s)


def _rope_table(s):
    c = s["case"]
    if own:
        from rank_latent_kv_gb300 import palu as P
        return P.rope_table(c["positions"], c["rope"], base=c["base"], scaling=c["kind"], factor=c["factor"],
                            original=c["original"], start=c["start"])
    freq, factor = _frequencies(c)
    f = torch.tensor(freq, dtype=torch.float64, device="cuda")
    ang = torch.arange(c["start"], c["start"] + c["positions"], dtype=torch.float64, device="cuda")[:, None] * f
    return (torch.cat([ang.cos(), ang.sin()], 1) * factor).float()


def _page_plan(s):
    """The new tokens' pages, then all of them refused: the lengths as before, and the pages given back."""
    if own:
        offsets, positions, slots = s["pool"].plan(s["new"], s["rows"])
        s["lengths"].copy_(s["before"])
        s["pool"].plan(s["none"], 0)
    else:
        offsets, positions, slots = _plan(s, s["new"], s["rows"])
        s["lengths"].copy_(s["before"])
        _plan(s, s["none"], 0)
    return {"offsets": offsets, "positions": positions, "slots": slots, "table": s["table"], "lengths": s["lengths"],
            "held": s["held"], "free": s["free"], "n_free": s["n_free"]}


def _plan(s, new, rows):
    page, table, held, free, n_free = s["case"]["page"], s["table"], s["held"], s["free"], s["n_free"]
    dev, old = table.device, s["lengths"].clone()
    total = old + new
    need = ((total + page - 1) // page).int()
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    col = torch.arange(table.shape[1], device=dev)
    # pages given back go on the stack, sequence by sequence
    at = n_free + (give.cumsum(0) - give)[:, None] + col - need[:, None]
    out = (col >= need[:, None]) & (col < held[:, None])
    stack = torch.cat([free, free.new_zeros(1)])
    stack[torch.where(out, at, free.shape[0]).flatten().long()] = table.flatten()
    free.copy_(stack[:-1])
    top = n_free + give.sum()
    # pages taken come off its top, sequence by sequence
    at = top - 1 - (take.cumsum(0) - take)[:, None] - (col - held[:, None])
    into = (col >= held[:, None]) & (col < need[:, None])
    table.copy_(torch.where(into, free[at.clamp(0, free.shape[0] - 1).long()], table))
    n_free.copy_(top - take.sum())
    held.copy_(need)
    s["lengths"].copy_(total)
    offsets = torch.cat([new.new_zeros(1), new.cumsum(0).int()])
    row = torch.arange(rows, device=dev)
    seq = torch.searchsorted(offsets[1:].long(), row, right=True).clamp(max=new.shape[0] - 1)
    pos = old[seq] + row - offsets[seq]
    slots = table[seq, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    there = row < offsets[-1]
    return offsets, torch.where(there, pos, -1), torch.where(there, slots, -1)


def _norm_rotate(x, weight, cos_sin, interleaved):
    """x [..., heads, D]: the norm of each head's row where there is a weight, then the rotation by cos_sin [..., rope]."""
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rope = cos_sin.shape[-1]
    cos, sin = cos_sin[..., None, :rope // 2], cos_sin[..., None, rope // 2:]
    if interleaved:
        a, b = x[..., 0:rope:2], x[..., 1:rope:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rope // 2], x[..., rope // 2:rope]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rope:]], -1)


def _places(s, n):
    """Of each of the n new tokens: its sequence, and its position in it."""
    at = torch.arange(n, device=s["q"].device)
    seq = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return seq, s["lengths"][seq] - s["offsets"][1:].long()[seq] + at


def _append4(s):
    c, n = s["case"], s["q"].shape[0]
    if own:
        q = s["cache"].append(s["k"], s["v"], s["offsets"], q=s["q"], cos_sin=s["cos_sin"], q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        k, v = s["cache"].read(s["offsets"], n)
        return {"q": q, "k": k, "v": v}
    dt, page = DTYPES[c["dtype"]], c["page"]
    seq, pos = _places(s, n)
    cs = s["cos_sin"][pos]
    q = _norm_rotate(s["q"], s["q_weight"], cs, c["interleaved"]).to(dt)
    k = _norm_rotate(s["k"], s["k_weight"], cs, c["interleaved"]).to(dt)
    ids, blk, tok = s["table"][seq, pos // page].long(), pos % page // 16, pos % 16
    kc, ks, vc, vs = _fields(s["pages"])
    codes, sc, z = _quantise(k.float())
    kc[ids, :, blk, tok] = _key_codes(codes)
    ks[ids, :, blk, tok] = torch.stack([sc, z], -2)
    codes, sc, z = _quantise(s["v"].float())
    pair, eight, odd = tok % 8 // 2, tok // 8, tok % 2
    vc[ids, :, blk, :, :, pair, :, 2 * odd + eight] = _value_codes(codes).transpose(-1, -2)
    vs[ids, :, blk, :, pair, eight, :, odd] = torch.stack([sc, z], -2)
    # and read back: key rows as they lie, the value rows out of their blocks
    k = _key_values(kc[ids, :, blk, tok], ks[ids, :, blk, tok]).to(dt)
    x = _nibbles(vc[ids, :, blk, :, :, pair, :, 2 * odd + eight])         # token head half g m nibble
    x = _move(x, 4, (0, 2, 3, 1)).flatten(-4).unflatten(-1, (4, G))
    sz = vs[ids, :, blk, :, pair, eight, :, odd].float()[..., None]
    v = (x.float() * sz[:, :, 0] + sz[:, :, 1]).flatten(-2).to(dt)
    return {"q": q, "k": k, "v": v}


def _attend4(s):
    c = s["case"]
    if own:
        return s["cache"].attend(s["q"], s["offsets"], s["max_new"], shared_pages=s["shared_pages"], workspace=s["workspace"])
    hq, hkv, page, t, sp = c["hq"], c["hkv"], c["page"], s["max_new"], s["shared_pages"]
    q, n, b, gq, shared = s["q"], s["q"].shape[0], c["batch"], hq // hkv, sp * page
    # the new tokens of every sequence, padded to the most that one has
    idx = s["offsets"][:-1].long()[:, None] + torch.arange(t, device=q.device)
    qp = q[idx.clamp(max=n - 1)].float().view(b, t, hkv, gq, D).permute(2, 0, 1, 3, 4)          # [hkv, b, t, gq, D]
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()
    pos = (s["lengths"] - count)[:, None] + torch.arange(t, device=q.device)                     # [b, t]

    def rows(ids, values):   # [..., ids, hkv, blocks, 16, D] -> [hkv, ..., tokens, D]
        kc, ks, vc, vs = _fields(s["pages"][ids.long()])
        x = _value_values(vc, vs) if values else _key_values(kc, ks)
        return x.movedim(-4, 0).flatten(-4, -2)

    own_ids, shared_ids = s["table"][:, sp:], s["table"][0, :sp]
    # scores over the shared prefix (one product for the batch), then over each sequence's own tokens
    sc = torch.cat([
        (qp.reshape(hkv, b * t * gq, D) @ rows(shared_ids, False).transpose(-1, -2)).view(hkv, b, t * gq, shared),
        qp.reshape(hkv, b, t * gq, D) @ rows(own_ids, False).transpose(-1, -2)], -1) / math.sqrt(D)
    sc = sc.view(hkv, b, t, gq, -1)
    seen = torch.arange(sc.shape[-1], device=q.device) <= pos[..., None]                         # [b, t, keys]
    sc = sc.masked_fill(~seen[None, :, :, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(hkv, b, t * gq, -1)
    o = p[..., shared:] @ rows(own_ids, True)
    o += (p[..., :shared].reshape(hkv, b * t * gq, shared) @ rows(shared_ids, True)).view(o.shape)
    o = o.view(hkv, b, t, gq, D).permute(1, 2, 0, 3, 4).reshape(b, t, hq, D)
    at = torch.arange(n, device=q.device)
    seq = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return o[seq, at - s["offsets"].long()[seq]].to(DTYPES[c["dtype"]])


# ------------------------------------------------------------------ the definition, in 64 bits

def _turn64(x, weight, angles, interleaved):
    """One token's heads [heads, D] in fp64: y = x / rms(x) * w, then each pair (i, j) turned by its angle's cos and sin."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(0.5)
    rope = angles.shape[-1]
    i = torch.arange(rope // 2, device=x.device)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + rope // 2)
    co, si = angles[..., None, :rope // 2].double(), angles[..., None, rope // 2:].double()
    y = x.clone()
    y[..., i] = x[..., i] * co - x[..., j] * si
    y[..., j] = x[..., i] * si + x[..., j] * co
    return y


def _held64(x):
    """What rows [..., 128] of the cache's type read back as, from codes taken in 64 bits."""
    x = x.double().reshape(*x.shape[:-1], 4, G)
    z = x.min(-1, keepdim=True).values.half().double()
    s = ((x.max(-1, keepdim=True).values - x.min(-1, keepdim=True).values) / 15).half().double()
    return (z + s * ((x - z) / s).nan_to_num(0.0, 15.0, 0.0).round().clamp(0, 15)).reshape(*x.shape[:-2], D)


def _one64(block, token, values):
    """Place by place: the 128 values [..., 128] of one token of blocks [..., 2560] of bytes."""
    ch = torch.arange(D, device=block.device)
    if values:
        g, hi, m, half = ch % 8, ch // 8 % 2, ch // 16 % 4, ch // 64
        byte = 1280 + 512 * half + 64 * g + 16 * (token % 8 // 2) + 4 * m + 2 * (token % 2) + token // 8
        nib = hi
        place = 2304 + 2 * (((token % 8 // 2 * 2 + token // 8) * 4 + ch // G) * 2 + token % 2)
        place_z = place + 128
    else:
        in8 = ch % 8
        n = in8 // 2 + 4 * (in8 % 2)
        byte, nib = 64 * token + 16 * (ch % G // 8) + 4 * (ch // G) + n // 2, n % 2
        place = 1024 + 16 * token + 2 * (ch // G)
        place_z = place + 8
    code = (block[..., byte].long() >> (4 * nib)) & 15
    s, z = (torch.stack([block[..., p], block[..., p + 1]], -1).view(torch.float16)[..., 0].double() for p in (place, place_z))
    return z + s * code


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "page_plan":
        return None                                   # whole numbers
    if op == "rope_table":
        freq, factor = _frequencies(s["case"])
        # e^(i p f) as the power of a power: p = 1024 a + b
        turn = torch.tensor(freq, dtype=torch.float64, device="cuda")
        p = torch.arange(case["start"], case["start"] + case["positions"], device="cuda")
        far, near = (torch.polar(torch.ones_like(x), x) for x in ((p // 1024 * 1024).double()[:, None] * turn,
                                                                  (p % 1024).double()[:, None] * turn))
        e = far * near * factor
        return torch.cat([e.real, e.imag], 1)
    new, lengths = _lengths(case)
    start = np.concatenate([[0], np.cumsum(new)])
    page = case["page"]
    if op == "append4":
        dt = DTYPES[case["dtype"]]
        out = {x: torch.empty(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"}
        for b, (n, length) in enumerate(zip(new, lengths)):
            span = slice(int(start[b]), int(start[b + 1]))
            ang = s["cos_sin"][torch.arange(length - n, length, device="cuda")]
            out["q"][span] = _turn64(s["q"][span], s["q_weight"], ang, case["interleaved"])
            # a key is held as its codes would hold the row that an uncompressed page holds
            out["k"][span] = _held64(_turn64(s["k"][span], s["k_weight"], ang, case["interleaved"]).float().to(dt))
            out["v"][span] = _held64(s["v"][span])
        return out
    if work(case)["flops"] > 1e12:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    gq = case["hq"] // case["hkv"]
    for b, (n, length) in enumerate(zip(new, lengths)):
        ids = s["table"][b].long()
        for h in range(case["hkv"]):
            blocks = s["pages"][ids, h].reshape(-1, BLOCK)
            k, v = (torch.stack([_one64(blocks, t, values) for t in range(16)], 1).reshape(-1, D)[:length]
                    for values in (False, True))
            q = s["q"][int(start[b]):int(start[b + 1]), h * gq:(h + 1) * gq].double().reshape(n * gq, D)
            sc = (q @ k.T) * D ** -0.5
            last = length - n + torch.arange(n, device=q.device).repeat_interleave(gq)
            sc[torch.arange(length, device=q.device)[None] > last[:, None]] = -math.inf
            out[int(start[b]):int(start[b + 1]), h * gq:(h + 1) * gq] = (torch.softmax(sc, -1) @ v).view(n, gq, D)
    return out
