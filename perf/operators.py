"""The serving operators of the paged cache, as cases to be measured.

Four operators of one serving step with drafted tokens, in the order in which
a program calls them: queries and keys normalised per head and rotated
(`qk_norm_rope`), new tokens appended to a paged key/value cache with the same
norm and rotation on the way (`append`), attention of the new tokens over the
paged cache with a prefix that the batch shares read once (`attend`), and the
verification of the drafted tokens against the target's probabilities
(`verify`).

`run` computes them in plain torch where `own` is false and calls the
package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

D = 128                     # head dimension of the framework
EPS = 1e-6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 16 sequences, 28 query and 4 KV heads: the smallest call, latency counts
        dict(name="norm_rope_step", op="qk_norm_rope", dtype="bf16", batch=16, tokens=1, hq=28, hkv=4, rope=128,
             interleaved=False, norm=True),
        # the prefill of four prompts before the latent caches are fitted, 24 query and 8 KV heads
        dict(name="norm_rope_prefill", op="qk_norm_rope", dtype="fp16", batch=4, tokens=4096, hq=24, hkv=8, rope=128,
             interleaved=False, norm=True),
        # one decode step's tokens into pages of 64
        dict(name="append_step", op="append", dtype="bf16", batch=16, new=1, ragged=False, length=4096, page=64,
             hq=28, hkv=4, rope=128, interleaved=False, norm=True),
        # prompt chunks of different lengths in one batch, interleaved pairs on half of the channels, no norm
        dict(name="append_chunks", op="append", dtype="fp16", batch=32, new=611, ragged=True, length=1500, page=16,
             hq=24, hkv=8, rope=64, interleaved=True, norm=False),
        # a single sequence's decode step: latency
        dict(name="attend_one", op="attend", dtype="fp16", batch=1, new=1, ragged=False, shared=0, own=513, page=16,
             hq=24, hkv=8),
        # 16 sequences of up to 32768 tokens, nothing shared: the cache read at memory speed
        dict(name="attend_long", op="attend", dtype="bf16", batch=16, new=1, ragged=False, shared=0, own=32768, page=64,
             hq=28, hkv=4),
        # decode of 32 sequences behind one 8192-token prompt
        dict(name="attend_shared_step", op="attend", dtype="fp16", batch=32, new=1, ragged=False, shared=8192, own=777,
             page=32, hq=24, hkv=8),
        # up to 5 tokens (one sampled, four drafted) of 64 sequences behind one 32768-token prompt
        dict(name="attend_shared_drafts", op="attend", dtype="bf16", batch=64, new=5, ragged=True, shared=32768, own=1024,
             page=64, hq=28, hkv=4),
        # prompt chunks of up to 512 tokens over a cache of 8192
        dict(name="attend_chunks", op="attend", dtype="bf16", batch=4, new=512, ragged=True, shared=0, own=8192, page=128,
             hq=24, hkv=8),
        # one sequence with four drafted tokens
        dict(name="verify_one", op="verify", batch=1, drafts=4, vocab=32000, ragged=False, draft_probs=True),
        # 64 sequences with up to seven drafted tokens, a large odd vocabulary
        dict(name="verify_batch", op="verify", batch=64, drafts=7, vocab=152065, ragged=True, draft_probs=True),
        # drafts copied from the prompt: no draft probabilities
        dict(name="verify_copied", op="verify", batch=16, drafts=3, vocab=65537, ragged=False, draft_probs=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((24, 8), (28, 4), (32, 8), (16, 16), (8, 1), (5, 1), (12, 4))


def draw(rng):
    op = rng.choice(("qk_norm_rope", "append", "attend", "attend", "attend", "verify"))
    hq, hkv = rng.choice(HEADS)
    dtype = rng.choice(("fp16", "bf16"))
    if op == "verify":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 152065),
                    ragged=rng.random() < 0.5, draft_probs=rng.random() < 0.7)
    pairs = dict(rope=rng.choice((32, 64, 128)), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6)
    if op == "qk_norm_rope":
        batch = _log(rng, 1, 32)
        return dict(op=op, dtype=dtype, batch=batch, tokens=_log(rng, 1, max(1, 16384 // batch)), hq=hq, hkv=hkv, **pairs)
    page = rng.choice((16, 32, 64, 128))
    batch = _log(rng, 1, 64)
    if op == "append":
        new = _log(rng, 1, max(1, 16384 // batch))
        return dict(op=op, dtype=dtype, batch=batch, new=new, ragged=rng.random() < 0.5,
                    length=new + _log(rng, 1, max(2, 65536 // batch)), page=page, hq=hq, hkv=hkv, **pairs)
    new = rng.choice((1, 1, 2, 3, 5, 8, 17, 64))
    new = min(new, max(1, 512 // batch))
    shared = rng.choice((0, 1, 1)) * (_log(rng, 128, 32768) // page) * page
    most = max(64, min(32768, (400000 if new <= 8 else 100000) // batch))
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
    if case["op"] == "append":
        return new, _own_lengths(case, case["length"], new)
    return new, [case["shared"] + x for x in _own_lengths(case, case["own"], new)]


def _n_drafts(case):
    b, k = case["batch"], case["drafts"]
    return [(k - i * 5 % (k + 1)) if case["ragged"] else k for i in range(b)]


def work(case):
    op = case["op"]
    if op == "verify":
        # the drafted tokens' probabilities, one row of each table a sequence, the answers
        b, k, rows = case["batch"], case["drafts"], 2 if case["draft_probs"] else 1
        return {"bytes": b * (rows * case["vocab"] * 4 + k * (8 + 4 + 4 * rows) + 4 + (k + 1) * 8 + 4 + 16),
                "flops": b * rows * case["vocab"]}
    hq, hkv = case["hq"], case["hkv"]
    if op == "qk_norm_rope":
        n = case["batch"] * case["tokens"]
        return {"bytes": n * (2 * (hq + hkv) * D * 2 + 8 + 4 * case["rope"]), "flops": n * (hq + hkv) * D * 8}
    new, lengths = _lengths(case)
    n = sum(new)
    if op == "append":
        return {"bytes": n * (2 * (hq + 2 * hkv) * D * 2 + 4 * case["rope"]), "flops": n * (hq + hkv) * D * 8}
    shared = case["shared"]
    keys = shared + sum(x - shared for x in lengths)
    # query t of a sequence sees the tokens up to its own
    pairs = sum(t * x - t * (t - 1) // 2 for t, x in zip(new, lengths))
    return {"bytes": keys * hkv * 2 * D * 2 + n * hq * 2 * D * 2, "flops": pairs * hq * 4 * D}


# ------------------------------------------------------------------ inputs

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


def _table(g, dev, rows, n_pages):
    """Page ids [rows] in no order, as an allocator hands them out after a while."""
    return torch.randperm(n_pages, generator=g, device=dev)[:rows].to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    op = case["op"]
    if op == "verify":
        return _prepare_verify(case, g, dev)
    dt, hq, hkv = DTYPES[case["dtype"]], case["hq"], case["hkv"]
    if op == "qk_norm_rope":
        b, t = case["batch"], case["tokens"]
        # queries, keys and values of the projection, one row a token
        qkv = torch.randn(b, t, hq + 2 * hkv, D, generator=g, device=dev).to(dt)
        start = torch.randint(0, 4096, (b, 1), generator=g, device=dev)
        s = {"op": op, "case": case, "q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hkv],
             "positions": start + torch.arange(t, device=dev)}
        s.update(_pairs_state(case, g, dev, 4096 + t))
        return s
    new, lengths = _lengths(case)
    b, page, n = case["batch"], case["page"], sum(new)
    shared_pages = case.get("shared", 0) // page
    own_pages = -(-(max(lengths) - shared_pages * page) // page)
    n_pages = shared_pages + b * own_pages + 3
    ids = _table(g, dev, shared_pages + b * own_pages, n_pages)
    table = torch.cat([ids[:shared_pages].expand(b, -1), ids[shared_pages:].view(b, own_pages)], 1).contiguous()
    mean = 0.5 * torch.randn(hkv, 1, D, generator=g, device=dev)        # keys and values have a mean a channel
    s = {"op": op, "case": case, "table": table, "shared_pages": shared_pages, "own_pages": own_pages,
         "lengths": torch.tensor(lengths, dtype=torch.int64, device=dev),
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev), "max_new": max(new),
         "k_pages": torch.empty(n_pages, hkv, page, D, dtype=dt, device=dev),
         "v_pages": torch.empty(n_pages, hkv, page, D, dtype=dt, device=dev)}
    for pages in (s["k_pages"], s["v_pages"]):
        for i in range(0, n_pages, 4096):                                 # in pieces: the fp32 normals are twice as large
            part = pages[i:i + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device=dev) + mean)
    if op == "append":
        qkv = torch.randn(n, hq + 2 * hkv, D, generator=g, device=dev).to(dt)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        s.update(_pairs_state(case, g, dev, max(lengths)))
    else:
        s["q"] = torch.randn(n, hq, D, generator=g, device=dev).to(dt)
    if own:  # the handle on the pages, and the attention's workspace, as a program keeps them
        from rank_latent_kv_gb300 import palu as P
        s["cache"] = P.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lengths"])
        if op == "attend":
            s["workspace"] = s["cache"].attend_workspace(n, hq, s["max_new"], shared_pages)
    return s


def _prepare_verify(case, g, dev):
    b, k, v = case["batch"], case["drafts"], case["vocab"]
    logits = 3.0 * torch.randn(b, k + 1, v, generator=g, device=dev)
    s = {"op": "verify", "case": case, "target": torch.softmax(logits, -1), "draft": None}
    if case["draft_probs"]:
        near = logits[:, :k] + torch.randn(b, k, v, generator=g, device=dev)     # a draft model near the target's
        s["draft"] = torch.softmax(near, -1)
        del near
    del logits
    pick = s["draft"] if s["draft"] is not None else s["target"][:, :k]
    s["tokens"] = torch.multinomial(pick.reshape(b * k, v), 1, generator=g).view(b, k)
    s["accept_u"] = torch.rand(b, k, generator=g, device=dev)
    s["sample_u"] = torch.rand(b, generator=g, device=dev)
    s["n_drafts"] = torch.tensor(_n_drafts(case), dtype=torch.int32, device=dev)
    s["lengths"] = 100 + k + torch.arange(b, device=dev, dtype=torch.int64)       # the cache's, drafts among them
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"qk_norm_rope": _qk_norm_rope, "append": _append, "attend": _attend, "verify": _verify}[s["op"]](s)


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


def _qk_norm_rope(s):
    c = s["case"]
    if own:
        from rank_latent_kv_gb300 import palu as P
        return P.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                              eps=EPS, interleaved=c["interleaved"])
    cs = s["cos_sin"][s["positions"]]
    q = _norm_rotate(s["q"], s["q_weight"], cs, c["interleaved"])
    k = _norm_rotate(s["k"], s["k_weight"], cs, c["interleaved"])
    return tuple(x.transpose(1, 2).to(DTYPES[c["dtype"]]).contiguous() for x in (q, k))


def _places(s, n):
    """Of each of the n new tokens: its sequence, and its position in it."""
    at = torch.arange(n, device=s["q"].device)
    seq = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return seq, s["lengths"][seq] - s["offsets"][1:].long()[seq] + at


def _append(s):
    c = s["case"]
    if own:
        q = s["cache"].append(s["k"], s["v"], s["offsets"], q=s["q"], cos_sin=s["cos_sin"], q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    dt, page = DTYPES[c["dtype"]], c["page"]
    seq, pos = _places(s, s["q"].shape[0])
    cs = s["cos_sin"][pos]
    q = _norm_rotate(s["q"], s["q_weight"], cs, c["interleaved"]).to(dt)
    k = _norm_rotate(s["k"], s["k_weight"], cs, c["interleaved"]).to(dt)
    ids = s["table"][seq, pos // page].long()
    s["k_pages"][ids, :, pos % page] = k
    s["v_pages"][ids, :, pos % page] = s["v"]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attend(s):
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

    def rows(pages, ids):   # [..., ids, hkv, page, D] -> [hkv, ..., ids * page, D]
        x = pages[ids.long()].float()
        return x.movedim(-3, 0).flatten(-3, -2)

    own_ids = s["table"][:, sp:]
    # scores over the shared prefix (one product for the batch), then over each sequence's own tokens
    sc = torch.cat([
        (qp.reshape(hkv, b * t * gq, D) @ rows(s["k_pages"], s["table"][0, :sp]).transpose(-1, -2)).view(hkv, b, t * gq, shared),
        qp.reshape(hkv, b, t * gq, D) @ rows(s["k_pages"], own_ids).transpose(-1, -2)], -1) / math.sqrt(D)
    sc = sc.view(hkv, b, t, gq, -1)
    seen = torch.arange(sc.shape[-1], device=q.device) <= pos[..., None]                         # [b, t, keys]
    sc = sc.masked_fill(~seen[None, :, :, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(hkv, b, t * gq, -1)
    v_own = rows(s["v_pages"], own_ids)
    o = p[..., shared:] @ v_own
    o += (p[..., :shared].reshape(hkv, b * t * gq, shared) @ rows(s["v_pages"], s["table"][0, :sp])).view(o.shape)
    o = o.view(hkv, b, t, gq, D).permute(1, 2, 0, 3, 4).reshape(b, t, hq, D)
    at = torch.arange(n, device=q.device)
    seq = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return o[seq, at - s["offsets"].long()[seq]].to(DTYPES[c["dtype"]])


def _verify(s):
    if own:
        from rank_latent_kv_gb300 import palu as P
        return P.draft_verify(s["target"], s["draft"], s["tokens"], s["accept_u"], s["sample_u"], n_drafts=s["n_drafts"],
                              lengths=s["lengths"])
    target, draft, tokens = s["target"], s["draft"], s["tokens"]
    b, k = tokens.shape
    n = s["n_drafts"].long()
    rows = torch.arange(b, device=target.device)
    p = target[:, :k].gather(2, tokens[..., None])[..., 0].double()
    q = draft.gather(2, tokens[..., None])[..., 0].double() if draft is not None else torch.ones_like(p)
    # a draft is kept while u q(x) < p(x) has held for it and for all before it
    kept = (s["accept_u"].double() * q < p) & (torch.arange(k, device=target.device) < n[:, None])
    n_acc = kept.long().cumprod(1).sum(1)
    # then one token from what the target has over the draft, or from the target behind the last draft
    weight = target[rows, n_acc].double()
    at = n_acc.clamp(max=k - 1)
    refused = (n_acc < n)[:, None]
    if draft is not None:
        over = (weight - draft[rows, at].double()).clamp(min=0)
    else:
        over = weight.scatter(1, tokens[rows, at][:, None], 0.0)
    over = torch.where(refused, over, weight)
    weight = torch.where(over.sum(1, keepdim=True) > 0, over, weight)
    total = weight.cumsum(1)
    token = (total <= s["sample_u"].double()[:, None] * total[:, -1:]).sum(1)
    col = torch.arange(k + 1, device=target.device)
    out = torch.cat([tokens, torch.full((b, 1), -1, device=target.device)], 1)
    out = torch.where(col < n_acc[:, None], out, torch.where(col == n_acc[:, None], token[:, None], -1))
    return out, n_acc.int(), s["lengths"] - (n - n_acc)


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


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None                                   # whole numbers
    if op == "qk_norm_rope":
        ang = s["cos_sin"][s["positions"]]
        return tuple(_turn64(s[x], s[x + "_weight"], ang, case["interleaved"]).permute(0, 2, 1, 3).contiguous() for x in "qk")
    new, lengths = _lengths(case)
    start = np.concatenate([[0], np.cumsum(new)])
    page = case["page"]
    if op == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        q = torch.empty(s["q"].shape, dtype=torch.float64, device=kp.device)
        for b, (n, length) in enumerate(zip(new, lengths)):
            span = slice(int(start[b]), int(start[b + 1]))
            pos = torch.arange(length - n, length, device=kp.device)
            ang = s["cos_sin"][pos]
            q[span] = _turn64(s["q"][span], s["q_weight"], ang, case["interleaved"])
            where = s["table"][b].long()[pos // page], slice(None), pos % page
            kp[where] = _turn64(s["k"][span], s["k_weight"], ang, case["interleaved"])
            vp[where] = s["v"][span].double()
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if work(case)["flops"] > 4e12:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    gq = case["hq"] // case["hkv"]
    for b, (n, length) in enumerate(zip(new, lengths)):
        ids = s["table"][b].long()
        for h in range(case["hkv"]):
            k = s["k_pages"][ids, h].reshape(-1, D)[:length].double()
            v = s["v_pages"][ids, h].reshape(-1, D)[:length].double()
            q = s["q"][int(start[b]):int(start[b + 1]), h * gq:(h + 1) * gq].double().reshape(n * gq, D)
            sc = (q @ k.T) * D ** -0.5
            last = length - n + torch.arange(n, device=q.device).repeat_interleave(gq)
            sc[torch.arange(length, device=q.device)[None] > last[:, None]] = -math.inf
            out[int(start[b]):int(start[b + 1]), h * gq:(h + 1) * gq] = (torch.softmax(sc, -1) @ v).view(n, gq, D)
    return out
