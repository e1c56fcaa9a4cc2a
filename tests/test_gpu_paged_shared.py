"""Attention behind a shared prefix, at sizes for which the shared pages are read
once.  That they were is part of each test: in a second call the other
sequences' leading table entries name a page of NaN, which only a call that
reads row 0's pages leaves out of its result.  Bars as in test_gpu_paged.py."""
import math

import pytest
import torch

from test_gpu_draft import inputs as verify_inputs, reference as verify_reference
from test_gpu_paged import D, DEV, DT, _table, attend_close, close, make_cache, offsets_of, ref_attend, ref_transform

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


def ref_by_sequence(q, pools, ids, lengths, new, page):
    """What ref_attend computes, a sequence at a time on the GPU in fp64 (longer calls)."""
    out, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    G, row = q.shape[1] // pools[0].shape[1], 0
    for b, n in enumerate(new):
        if n and lengths[b]:
            t = torch.arange(lengths[b])
            at = ids[b].cpu().long()[t // page], slice(None), t % page
            k, v = (x[at].to(DEV).double().repeat_interleave(G, 1).transpose(0, 1) for x in pools)      # [Hq, len, D]
            s = q[row:row + n].to(DEV).double().transpose(0, 1) @ k.transpose(1, 2) / math.sqrt(D)      # [Hq, n, len]
            lim = lengths[b] - n + 1 + torch.arange(n, device=DEV)
            p = torch.softmax(s.masked_fill(t.to(DEV) >= lim[:, None], -math.inf), -1).nan_to_num(0.0)   # nothing seen: zeros
            out[row:row + n], mag[row:row + n] = (p @ v).transpose(0, 1).cpu(), (p @ v.abs()).transpose(0, 1).cpu()
        row += n
    return out, mag


def hide_shared(c, dev, shared):
    """Rows 1.. of the table name a page of NaN for the shared pages; returns the table as it was."""
    was = c.page_table.clone()
    free = sorted(set(range(dev[0].shape[0])) - set(was.flatten().tolist()))[0]
    for t in dev:
        t[free] = NAN
    c.page_table[1:, :shared] = free
    return was


BEHIND = [  # page, new, lengths, Hq, Hk, shared pages, table width: no sequence as long as the named prefix
    (16, [1] * 8, [100 + 17 * i for i in range(8)], 64, 64, 16, 16),          # up to 8 rows, two launches' sizes or one
    (16, [1] * 8, [1 + 16 * i for i in range(8)], 64, 64, 32, 100),           # whole tiles that nobody sees
    (64, [2, 0, 1, 2, 2, 1, 0, 2], [190, 300, 0, 129, 128, 127, 1, 191], 64, 64, 8, 30),  # 10 rows; the longest has none
    (128, [1] * 30, [1 + 8 * i for i in range(30)], 64, 32, 2, 2),            # many rows, one launch
    (32, [1] * 30, [200 + i for i in range(30)], 64, 32, 8, 60),              # many rows, own keys on few
    (64, [20, 20, 1, 7, 20, 3, 0, 20], [300, 132, 200, 115, 300, 13, 10, 60], 96, 96, 8, 12),  # many rows throughout
]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,shared,width", BEHIND)
def test_what_lies_behind_all_lengths_does_not_matter(P, dt, page, new, lengths, Hq, Hk, shared, width):
    """Every sequence ends inside the named prefix (a fixed number of pages in a captured graph, after a rollback); NaN
    behind the longest that has new rows."""
    d = DT[dt]
    seen = [l if m else 0 for l, m in zip(lengths, new)]
    pools, dev, c = make_cache(P, d, seen, page, Hk, seed=page + sum(lengths), shared=shared, width=width, fill=NAN)
    c.lengths.copy_(torch.tensor(lengths))
    n = sum(new)
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(n)).to(d)
    ref, mag = ref_attend(q, pools, c.page_table.cpu(), lengths, new, page)
    a = c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared)
    assert c.sync() == 0
    attend_close(a, ref, mag, d)
    hide_shared(c, dev, shared)
    b = c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared)
    assert c.sync() == 0 and torch.equal(a, b)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,shared", [
    (16, [1] * 8, [520 + 90 * i for i in range(8)], 64, 64, 32),              # up to 8 rows: one line
    (32, [1] * 30, [400 + 60 * i for i in range(30)], 96, 32, 8),             # many rows and few, Gq 3
    (64, [2, 2, 1, 2, 2, 0, 2, 1] * 3, [900 + 40 * i for i in range(24)], 112, 16, 13),  # the same, Gq 7, 14 rows
    (128, [6] * 24, [1550 + 30 * i for i in range(24)], 24, 8, 12),           # many rows throughout
])
def test_the_tables_width_is_not_the_lengths(P, dt, page, new, lengths, Hq, Hk, shared):
    """A program's table is as wide as the longest sequence that it admits.  How a call's work is divided follows from the
    lengths, so the same call in a table of 131,072 tokens gives the same bits as in one cut to the lengths."""
    d = DT[dt]
    pools, dev, c = make_cache(P, d, lengths, page, Hk, seed=sum(lengths), shared=shared, fill=NAN)
    n = sum(new)
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(n)).to(d)
    ref, mag = ref_by_sequence(q, pools, c.page_table.cpu(), lengths, new, page)
    was = hide_shared(c, dev, shared)
    out = [c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared)]
    assert c.sync() == 0
    attend_close(out[0], ref, mag, d)
    for tokens in (1 << 13, 1 << 17):
        wide = torch.full((len(new), tokens // page), -1, dtype=torch.int32, device=DEV)   # behind the lengths: no page
        wide[:, :was.shape[1]] = c.page_table
        w = P.PagedCache(dev[0], dev[1], wide, c.lengths)
        out.append(w.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared))
        assert w.sync() == 0
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


# Calls that share: up to 16 rows in all (one line of the few-rows kernel); many rows and own units of few, with 3 and 7
# query heads a KV head, so that row tiles begin inside a token; many rows throughout, in own units of one and of several
# row tiles.
KINDS = {  # page, new, Hq, Hk, shared pages, pages a sequence may have of its own
    "few": (16, [2, 2, 1, 2, 0, 2, 2, 2], 16, 16, 64, 20),
    "both": (32, [1, 0, 1, 1] * 8, 24, 8, 64, 12),
    "both7": (64, [2, 2, 1, 2, 2, 0, 2, 1] * 6, 28, 4, 40, 8),
    "many": (128, [6, 5, 6, 1, 6, 6, 0, 6] * 4, 24, 8, 12, 5),
    "tall": (64, [38, 37, 40, 0] * 4, 28, 4, 160, 4),
}


def kind_lengths(kind, seed):
    """Own tokens of every number, none included; sequences that end at, and just behind, the prefix, and inside it."""
    page, new, Hq, Hk, shared, own = KINDS[kind]
    g = torch.Generator().manual_seed(seed)
    S0 = page * shared
    lengths = [S0 + int(torch.randint(n, own * page + 1, (1,), generator=g)) for n in new]
    for b, l in ((1, S0), (2, S0 + 1), (4, S0 - 1), (5, S0 // 3), (7, 1 if seed % 2 else 0)):
        lengths[b] = l
    return lengths


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_every_kind_of_shared_call(P, dt, kind):
    """Against 64 bits, with rows behind the last sequence, NaN behind all lengths and anything in the workspace."""
    page, new, Hq, Hk, shared, own = KINDS[kind]
    d, lengths, n = DT[dt], kind_lengths(kind, 1), sum(new)
    pools, dev, c = make_cache(P, d, lengths, page, Hk, layout="tokens", seed=len(new), shared=shared, width=shared + own, fill=NAN)
    q = torch.randn(n + 2, Hq, D, generator=torch.Generator().manual_seed(n)).to(d)
    ref, mag = ref_by_sequence(q[:n], pools, c.page_table, lengths, new, page)
    ws = c.attend_workspace(n + 2, Hq, max(new), shared)
    out = []
    for fill in (0, 255):
        ws.fill_(fill)
        o = torch.full((n + 2, Hq, D), 7.0, dtype=d, device=DEV)
        c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared, workspace=ws, out=o)
        assert c.sync() == 0 and (o[n:] == 7).all()
        attend_close(o[:n], ref, mag, d)
        out.append(o)
        hide_shared(c, dev, shared)
    assert torch.equal(out[0], out[1])


def _word(P, c):
    with pytest.raises(P.PaluError) as e:
        c.sync()
    return int(str(e.value).split("word ")[1].split(":")[0])


@pytest.mark.parametrize("kind", KINDS)
def test_what_the_device_refuses_in_a_shared_call(P, kind):
    """Bad spans, rows before the first sequence, a length past the table, pages outside the pool: the error word, zeros
    where the header says so, and the other sequences served."""
    page, new, Hq, Hk, shared, own = KINDS[kind]
    d, lengths, most = torch.bfloat16, kind_lengths(kind, 2), max(new)
    pools, dev, c = make_cache(P, d, lengths, page, Hk, seed=3, shared=shared, width=shared + own)
    hide_shared(c, dev, shared)
    table, spare = c.page_table.clone(), c.lengths.clone()
    q = torch.randn(sum(new) + most + 5, Hq, D, generator=torch.Generator().manual_seed(4)).to(d)

    def attend(counts, first=0):
        end = first + sum(counts)
        out = torch.full((end + 1, Hq, D), 7.0, dtype=d, device=DEV)
        c.attend(q[:end + 1].to(DEV), offsets_of(counts) + first, most, shared_pages=shared, out=out)
        assert (out[end:] == 7).all() and (out[:first] == 0).all()
        return out[first:end], ref_by_sequence(q[first:end], pools, table0, lengths, counts, page)

    def served(out, ref, counts, but):
        row = 0
        for b, m in enumerate(counts):
            if m and b != but:
                attend_close(out[row:row + m], ref[0][row:row + m], ref[1][row:row + m], d)
            elif m:
                assert (out[row:row + m] == 0).all()
            row += m
    table0 = table.clone()
    table0[1:, :shared] = table[0, :shared]
    # a sequence with more rows than max_new
    counts = list(new)
    counts[3] = most + 1
    out, ref = attend(counts)
    assert _word(P, c) == P.PALU_DEVERR_SPAN
    served(out, ref, counts, 3)
    # rows before the first sequence
    out, ref = attend(new, first=3)
    assert _word(P, c) == P.PALU_DEVERR_SPAN
    served(out, ref, new, -1)
    # a length past the table is cut to it, the other sequences are served
    c.lengths[0] = 1 << 40
    out, ref = attend(new)
    assert _word(P, c) == P.PALU_DEVERR_CAPACITY and torch.isfinite(out[:new[0]]).all()
    m = new[0]
    attend_close(out[m:], ref[0][m:], ref[1][m:], d)
    c.lengths.copy_(spare)
    # an own page outside the pool: that sequence reads page 0, the others are served
    for bad in (-1, dev[0].shape[0], 0x7fffffff):
        c.page_table.copy_(table)
        c.page_table[0, shared] = bad
        out, ref = attend(new)
        assert _word(P, c) == P.PALU_DEVERR_PAGE
        attend_close(out[m:], ref[0][m:], ref[1][m:], d)
    # a shared one: no fault, and the word
    c.page_table.copy_(table)
    c.page_table[0, 1] = -5
    attend(new)
    assert _word(P, c) == P.PALU_DEVERR_PAGE
    c.page_table.copy_(table)
    out, ref = attend(new)
    assert c.sync() == 0
    served(out, ref, new, -1)


@pytest.mark.parametrize("kind", KINDS)
def test_shared_calls_between_copies_and_fills(P, kind):
    """Queries, lengths, offsets and pages copied right before the calls, results filled before and read right behind them;
    eagerly and in a captured graph that follows what the program writes."""
    page, new, Hq, Hk, shared, own = KINDS[kind]
    d, n = torch.float16, sum(new)
    lengths = [kind_lengths(kind, i) for i in range(4)]
    longest = [max(l) for l in zip(*lengths)]
    pools, dev, c = make_cache(P, d, longest, page, Hk, seed=5, shared=shared, width=shared + own)
    hide_shared(c, dev, shared)
    table0 = c.page_table.clone()
    table0[1:, :shared] = c.page_table[0, :shared]
    g = torch.Generator().manual_seed(6)
    src = torch.randn(4, n, Hq, D, generator=g).to(d).to(DEV)
    counts = [new, list(reversed(new)), new, [max(0, m - 1) for m in new]]
    all_lengths = torch.tensor([[max(l, 0) for l in x] for x in lengths], device=DEV)
    all_offsets = torch.stack([offsets_of(x) for x in counts])
    pick = torch.zeros(1, dtype=torch.int64, device=DEV)
    q, out, first = (torch.zeros(n, Hq, D, dtype=d, device=DEV) for _ in range(3))
    off = offsets_of(new)
    ws = c.attend_workspace(n, Hq, max(new), shared)

    def step():
        q.zero_()
        q.copy_(src[pick][0])
        c.lengths.copy_(all_lengths[pick][0])
        off.copy_(all_offsets[pick][0])
        out.fill_(7.0)
        c.attend(q, off, max(new), shared_pages=shared, workspace=ws, out=out)
        first.copy_(out)
        out.fill_(9.0)
        c.attend(q, off, max(new), shared_pages=shared, workspace=ws, out=out)

    def check(i):
        pick.fill_(i)
        run()
        a, b, m = first.clone(), out.clone(), sum(counts[i])
        assert c.sync() == 0 and torch.equal(a[:m], b[:m]) and (a[m:] == 7).all() and (b[m:] == 9).all()
        ref, mag = ref_by_sequence(src[i, :m].cpu(), pools, table0, lengths[i], counts[i], page)
        attend_close(a[:m], ref, mag, d)
    run = step
    for i in range(4):
        check(i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    run = graph.replay
    for i in (2, 0, 3, 1, 1, 2):
        check(i)


def test_shared_calls_on_several_streams(P):
    """Calls of every kind at once, each on a stream and with a workspace of its own."""
    calls = []
    for i, kind in enumerate(KINDS):
        page, new, Hq, Hk, shared, own = KINDS[kind]
        lengths = kind_lengths(kind, 3)
        pools, dev, c = make_cache(P, torch.bfloat16, lengths, page, Hk, seed=7, shared=shared, width=shared + own)
        table0 = c.page_table.clone()
        hide_shared(c, dev, shared)
        q = torch.randn(sum(new), Hq, D, generator=torch.Generator().manual_seed(i)).bfloat16()
        ref = ref_by_sequence(q, pools, table0, lengths, new, page)
        calls.append((c, q.to(DEV), offsets_of(new), max(new), shared, c.attend_workspace(len(q), Hq, max(new), shared),
                      torch.zeros_like(q, device=DEV), torch.cuda.Stream(), ref))
    torch.cuda.synchronize()
    for _ in range(6):
        for c, q, off, most, shared, ws, out, s, _ in calls:
            c.attend(q, off, most, shared_pages=shared, workspace=ws, out=out, stream=s)
    torch.cuda.synchronize()
    for c, q, off, most, shared, ws, out, s, ref in calls:
        assert c.sync() == 0
        attend_close(out, *ref, torch.bfloat16)


@pytest.mark.parametrize("dt,Hq,Hk,page,shared", [("fp16", 48, 16, 16, 128), ("bf16", 28, 4, 64, 64), ("bf16", 16, 16, 32, 40)])
def test_steps_behind_a_shared_prompt(P, dt, Hq, Hk, page, shared):
    """Steps of a loop with drafts: keys rotated and appended, attention behind the shared prompt, drafts verified, the
    lengths rolled back in place, the next step on what remains."""
    d, B, k, V, own = DT[dt], 20, 2, 211, 200 // page + 2
    g = torch.Generator().manual_seed(Hq + page)
    lengths = [page * shared + int(torch.randint(1, 100, (1,), generator=g)) for _ in range(B)]
    pools, dev, c = make_cache(P, d, lengths, page, Hk, seed=9, shared=shared, width=shared + own)
    table0 = c.page_table.clone()
    hide_shared(c, dev, shared)
    cs = _table(1 << 14, 128)
    csd = cs.to(DEV)
    for step in range(4):
        drafts = torch.randint(0, k + 1, (B,), generator=g)
        new = [int(x) + 1 for x in drafts]
        n = sum(new)
        c.lengths += torch.tensor(new, device=DEV)
        lengths = c.lengths.tolist()
        x = torch.randn(n, Hq + 2 * Hk, D, generator=g).to(d)
        xd, off = x.to(DEV), offsets_of(new)
        q = c.append(xd[:, Hq:Hq + Hk], xd[:, Hq + Hk:], off, q=xd[:, :Hq], cos_sin=csd)
        out = c.attend(q, off, k + 1, shared_pages=shared)
        assert c.sync() == 0
        pos = torch.cat([torch.arange(l - m, l) for l, m in zip(lengths, new)])
        close(q, *ref_transform(x[:, :Hq], None, cs[pos], False, 1e-6), d)
        host = [t.cpu() for t in dev]
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
        at = table0.cpu().long()[seq, pos // page], slice(None), pos % page
        close(host[0][at], *ref_transform(x[:, Hq:Hq + Hk], None, cs[pos], False, 1e-6), d)
        assert torch.equal(host[1][at], x[:, Hq + Hk:])
        attend_close(out, *ref_by_sequence(q.cpu(), host, table0, lengths, new, page), d)
        t, p, tokens, au, su = verify_inputs(B, k, V, step, near=0.5)
        on = [torch.from_numpy(a).to(DEV) for a in (t, p, tokens, au, su)]
        toks, kept, _ = P.draft_verify(*on, n_drafts=drafts.int().to(DEV), lengths=c.lengths, new_lengths=c.lengths)
        rt, rk = verify_reference(t, p, tokens, au, su, drafts.numpy())
        assert (toks.cpu().numpy() == rt).all() and (kept.cpu().numpy() == rk).all()
        assert c.lengths.tolist() == [l - int(a) + int(b) for l, a, b in zip(lengths, drafts, rk)]


@pytest.mark.parametrize("kind", KINDS)
def test_no_new_tokens_behind_a_shared_prefix(P, kind):
    """A padded batch without any new token: nothing is read that matters, nothing is written."""
    page, new, Hq, Hk, shared, own = KINDS[kind]
    pools, dev, c = make_cache(P, torch.bfloat16, kind_lengths(kind, 1), page, Hk, seed=8, shared=shared, width=shared + own)
    n = sum(new)
    q = torch.full((n, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    c.attend(q, torch.zeros(len(new) + 1, dtype=torch.int32, device=DEV), max(new), shared_pages=shared, out=out)
    assert c.sync() == 0 and (out == 7).all()


@pytest.mark.parametrize("B,new,Hq,Hk,shared", [(1500, 1, 8, 2, 16), (900, 3, 6, 2, 40), (700, 5, 16, 2, 64)])
def test_more_sequences_than_a_cta_has_threads(P, B, new, Hq, Hk, shared):
    """Many short sequences behind a prefix: some without rows, some that end inside it, most with few own tokens."""
    page, d = 16, torch.float16
    g = torch.Generator().manual_seed(B)
    counts = torch.randint(0, new + 1, (B,), generator=g).tolist()
    counts[5], counts[B - 1] = new, new
    lengths = [page * shared + int(torch.randint(m, 80, (1,), generator=g)) for m in counts]
    for b in range(0, B, 50):
        lengths[b] = int(torch.randint(0, page * shared + 1, (1,), generator=g))
    pools, dev, c = make_cache(P, d, lengths, page, Hk, seed=10, shared=shared, width=shared + 5)
    table0 = c.page_table.clone()
    hide_shared(c, dev, shared)
    n = sum(counts)
    q = torch.randn(n, Hq, D, generator=g).to(d)
    out = c.attend(q.to(DEV), offsets_of(counts), new, shared_pages=shared)
    assert c.sync() == 0
    attend_close(out, *ref_by_sequence(q, pools, table0, lengths, counts, page), d)
