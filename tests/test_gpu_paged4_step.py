"""The 4-bit paged cache, planned pages and rotation tables as a program uses
them together: steps with prompts, drafts and rollback against 64 bits and
against the uncompressed cache's rows; and calls at the edges of the plan
(many sequences, shared prefixes that some sequences do not fill, none new).

The caches are filled by appends, whose bytes tests/test_gpu_paged4.py holds to
the format; the reference takes what the bytes stand for.  Bars: as there; here as a norm over
each output row (the bars' terms are sums over keys of independent roundings):
2e-3 of the row for fp16, and the output's own rounding, 2^-8 in all, for bf16.
"""
import math

import pytest
import torch

from oracle import paged4_oracle as O4

pytestmark = pytest.mark.gpu

DEV = "cuda"
D = 128
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
BAR = {torch.float16: 2e-3, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


def offsets_of(new):
    return torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=DEV)


def decode(blocks, values):
    """Blocks [..., 2560] -> what they stand for, [..., 16, 128] in 64 bits, place by place."""
    place, scale = (torch.from_numpy(O4.PLACES[i + 2 * values]).to(DEV) for i in (0, 1))
    codes = (blocks[..., place[..., 0]] >> place[..., 1].to(torch.uint8)) & 15
    s, z = (torch.stack([blocks[..., scale[..., i]], blocks[..., scale[..., i] + 1]], -1).view(torch.float16)[..., 0].double()
            for i in (0, 1))
    return codes.double() * s.repeat_interleave(32, -1) + z.repeat_interleave(32, -1)


def rows_of(cache, b, length):
    """Keys and values of one sequence, [length, Hk, 128] in 64 bits, from the pages' bytes."""
    ids = cache.page_table[b, :-(-length // cache.page_size)].long()
    blocks = cache.pages[ids].unflatten(-1, (-1, O4.BLOCK)).transpose(1, 2).flatten(0, 1)
    return [decode(blocks, v).transpose(1, 2).flatten(0, 1)[:length] for v in (False, True)]


def check(cache, q, new, out, lengths, only=None):
    gq = q.shape[1] // cache.kv_heads
    at = 0
    for b, n in enumerate(new):
        if n and lengths[b] and (only is None or b in only):
            k, v = (x.repeat_interleave(gq, 1) for x in rows_of(cache, b, lengths[b]))
            s = torch.einsum("nhd,thd->hnt", q[at:at + n].double(), k) * D ** -0.5
            seen = torch.arange(lengths[b], device=DEV)[None] <= (lengths[b] - n + torch.arange(n, device=DEV))[:, None]
            w = torch.softmax(s.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
            ref = torch.einsum("hnt,thd->nhd", w, v)
            err = (out[at:at + n].double() - ref).norm(dim=-1)
            assert bool((err <= BAR[cache.dtype] * ref.norm(dim=-1) + 1e-7).all()), (b, float((err / ref.norm(dim=-1)).max()))
        at += n


def filled(P, dt, B, Hk, page, length, shared=0, width=None, fill=0xFF, seed=0):
    """A cache of B sequences of `length` tokens each, the first `shared` pages the same for all."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = width or -(-length // page)
    own = width - shared
    n_pages = shared + B * own + 1
    ids = torch.randperm(n_pages, generator=g, device=DEV)[:shared + B * own].int()
    table = torch.cat([ids[:shared].expand(B, -1), ids[shared:].view(B, own)], 1).contiguous()
    pages = torch.full((n_pages, Hk, page * 160), fill, dtype=torch.uint8, device=DEV)
    lengths = torch.full((B,), length, dtype=torch.int64, device=DEV)
    cache = P.PagedCache4(pages, table, lengths, page, dt)
    one = P.PagedCache4(pages, table[:1].contiguous(), lengths[:1].clone(), page, dt)
    mean = torch.randn(2, Hk, D, generator=g, device=DEV) / 2
    kv = (torch.randn(length, 2, Hk, D, generator=g, device=DEV) + mean).to(dt)
    one.append(kv[:, 0], kv[:, 1], offsets_of([length]))                     # the shared pages, and sequence 0
    rest = length - shared * page
    if rest > 0:
        kv = (torch.randn(B * rest, 2, Hk, D, generator=g, device=DEV) + mean).to(dt)
        cache.append(kv[:, 0], kv[:, 1], offsets_of([rest] * B))
    return cache


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hk,page,scaling", [(24, 8, 16, "parts"), (28, 4, 64, "plain"), (5, 1, 32, "ntk")])
def test_speculative_steps(P, dt, Hq, Hk, page, scaling):
    """Prompts, then steps of up to four drafts: pages from the pool, tables for the rotation, appends, attention, drafts
    verified on the device and rolled back by their lengths; an uncompressed cache on the same plan says what rows are."""
    dt = DT[dt]
    B, width, n_pages = 3, 12, 40
    g = torch.Generator(device=DEV).manual_seed(Hq)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    lengths = torch.zeros(B, dtype=torch.int64, device=DEV)
    pool = P.PagePool(table, lengths, page, n_pages=n_pages)
    pages = torch.full((n_pages, Hk, P.PagedCache4.page_bytes(page)), 0xFF, dtype=torch.uint8, device=DEV)
    cache = P.PagedCache4(pages, table, lengths, page, dt)
    plain_pages = torch.zeros(2, n_pages, Hk, page, D, dtype=dt, device=DEV)
    plain = P.PagedCache(plain_pages[0], plain_pages[1], table, lengths)
    cos_sin = P.rope_table(width * page, D, scaling=scaling, factor=4.0, original=64)
    w = (1 + 0.2 * torch.randn(2, D, generator=g, device=DEV)).to(dt)
    N = 160
    for step, new in enumerate(([40, 1, 100], [5, 5, 5], [5, 0, 3], [1, 5, 5], [5, 5, 1], [2, 5, 4])):
        counts = torch.tensor(new, dtype=torch.int32, device=DEV)
        off, pos, slots = pool.plan(counts, N)
        assert off.tolist() == offsets_of(new).tolist() and pool.sync() == 0
        x = torch.randn(N, Hq + 2 * Hk, D, generator=g, device=DEV).to(dt)
        args = dict(q=x[:, :Hq], cos_sin=cos_sin, q_weight=w[0], k_weight=w[1])
        q = cache.append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], off, positions=pos.clamp(min=0), **args)
        q2 = plain.append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], off, **args)
        n = sum(new)
        assert torch.equal(q[:n], q2[:n])
        out = cache.attend(q, off, max(new))
        now = lengths.tolist()
        check(cache, q, new, out, now)
        # 4 bits a value: within a step of the range of 32 channels of what the uncompressed cache holds
        flat = [t.transpose(1, 2).reshape(-1, Hk, D)[slots[:n]] for t in plain_pages]
        for got, ref in zip(cache.read(off, n), flat):
            r = ref.float().view(n, Hk, 4, 32)
            step_size = (r.amax(-1, keepdim=True) - r.amin(-1, keepdim=True)) / 15
            assert bool(((got.float().view_as(r) - r).abs() <= 0.52 * step_size + 2.0 ** -8 * r.abs()).all())
        full = plain.attend(q, off, max(new))
        # 32 normals' range is about 4 deviations, a step 0.27, its error 0.08 of a value; the keys' moves a weight by as
        # much: 0.11 of the output in all, twice that at most
        assert float((out[:n].float() - full[:n].float()).norm() / full[:n].float().norm()) < 0.23
        # of each sequence's drafts (all but its first new token) some are kept
        drafts = torch.randint(0, 50, (B, 4), generator=g, device=DEV)
        p = torch.softmax(torch.randn(B, 5, 50, generator=g, device=DEV), -1)
        n_drafts = (counts - 1).clamp(0, 4)
        _, kept, left = P.draft_verify(p, None, drafts, torch.rand(B, 4, generator=g, device=DEV),
                                       torch.rand(B, generator=g, device=DEV), n_drafts=n_drafts, lengths=lengths)
        if step:
            lengths.copy_(left)
        assert cache.sync() == 0 and plain.sync() == 0
    lengths.zero_()
    pool.plan(torch.zeros(B, dtype=torch.int32, device=DEV), 0)
    assert pool.n_free.item() == n_pages and sorted(pool.free_pages.tolist()) == list(range(n_pages))


def test_a_captured_loop_crosses_pages(P):
    """Plan, append, attention in one graph: no word from the host while sequences grow over their pages' borders."""
    B, Hq, Hk, page, N = 4, 8, 2, 16, 8
    table, lengths = torch.zeros(B, 6, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int64, device=DEV)
    pool = P.PagePool(table, lengths, page, n_pages=24)
    pages = torch.zeros(24, Hk, 160 * page, dtype=torch.uint8, device=DEV)
    cache = P.PagedCache4(pages, table, lengths, page, torch.float16)
    counts = torch.zeros(B, dtype=torch.int32, device=DEV)
    x = torch.zeros(N, Hq + 2 * Hk, D, dtype=torch.float16, device=DEV)
    off, pos = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.int64, device=DEV)
    slots, q, out = torch.zeros_like(pos), torch.zeros(N, Hq, D, dtype=torch.float16, device=DEV), torch.zeros(N, Hq, D, dtype=torch.float16, device=DEV)
    ws = cache.attend_workspace(N, Hq, 2)

    def step():
        pool.plan(counts, N, offsets=off, positions=pos, slots=slots)
        cache.append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], off, q=x[:, :Hq], q_out=q)
        cache.attend(q, off, 2, workspace=ws, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    counts.copy_(torch.tensor([2, 1, 0, 2]))
    g = torch.Generator(device=DEV).manual_seed(0)
    for i in range(30):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        graph.replay()
        if i % 10 == 9:
            check(cache, q, [2, 1, 0, 2], out, [2 * i + 2, i + 1, 0, 2 * i + 2])
    assert cache.sync() == 0 and pool.sync() == 0 and pool.held.tolist() == [4, 2, 0, 4]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,Hq,Hk,page,shared,length,new", [
    (40, 24, 8, 32, 128, 4500, 1),       # a line each: prefix of many rows, own units of few
    (40, 32, 2, 64, 64, 4300, 1),        # own units of 16 rows
    (24, 28, 4, 64, 64, 4300, 5),        # many rows in both
    (4, 2, 1, 128, 32, 4200, 1)])        # few rows in both
def test_shared_prefix_with_sequences_that_do_not_fill_it(P, dt, B, Hq, Hk, page, shared, length, new):
    cache = filled(P, DT[dt], B, Hk, page, length, shared=shared)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(B * new, Hq, D, generator=g, device=DEV).to(DT[dt])
    off = offsets_of([new] * B)
    out = cache.attend(q, off, new, shared_pages=shared)
    some = (0, 1, B - 1)
    check(cache, q, [new] * B, out, [length] * B, only=some)
    alone = cache.attend(q, off, new)
    assert float((out.float() - alone.float()).norm() / alone.float().norm()) < BAR[DT[dt]]
    assert torch.equal(out, cache.attend(q, off, new, shared_pages=shared))
    # lengths inside the prefix, of nothing, and one that ends with it
    lengths = [length] * B
    lengths[1], lengths[2], lengths[-1] = shared * page // 2 + 3, 0, shared * page
    cache.lengths.copy_(torch.tensor(lengths))
    out = cache.attend(q, off, new, shared_pages=shared)
    check(cache, q, [new] * B, out, lengths, only=(0, 1, B - 1))
    assert bool((out[2 * new:3 * new] == 0).all()) and cache.sync() == 0
    # all of them shorter than the prefix: what lies behind the longest does not matter
    cut = shared * page - page // 2 - 7
    cache.lengths.fill_(cut)
    for b in (cut // page, cut // page + 1):
        if b < shared:
            blk = cache.pages[int(cache.page_table[0, b])].view(Hk, page // 16, 2560)
            first = (cut - b * page + 15) // 16 if b == cut // page else 0
            blk[:, first:] = 0xFF
    out = cache.attend(q, off, new, shared_pages=shared)
    assert bool(torch.isfinite(out).all())
    check(cache, q, [new] * B, out, [cut] * B, only=some)


@pytest.mark.parametrize("B,Hq,Hk,new", [(4096, 2, 1, 1), (1000, 8, 2, 1), (700, 7, 1, 3), (300, 12, 2, 5)])
def test_many_sequences(P, B, Hq, Hk, new):
    length = 37
    cache = filled(P, torch.float16, B, Hk, 16, length, seed=3)
    q = torch.randn(B * new, Hq, D, device=DEV).half()
    out = cache.attend(q, offsets_of([new] * B), new)
    check(cache, q, [new] * B, out, [length] * B, only=(0, 1, B // 2, B - 1))
    # all of them at once
    blocks = cache.pages[cache.page_table.long()].unflatten(-1, (-1, O4.BLOCK)).transpose(2, 3).flatten(1, 2)
    k, v = (decode(blocks, x).transpose(2, 3).flatten(1, 2)[:, :length].repeat_interleave(Hq // Hk, 2) for x in (False, True))
    s = torch.einsum("bnhd,bthd->bhnt", q.view(B, new, Hq, D).double(), k) * D ** -0.5
    seen = torch.arange(length, device=DEV)[None] <= (length - new + torch.arange(new, device=DEV))[:, None]
    ref = torch.einsum("bhnt,bthd->bnhd", torch.softmax(s.masked_fill(~seen, -math.inf), -1), v).reshape(B * new, Hq, D)
    assert float(((out.double() - ref).norm(dim=-1) / ref.norm(dim=-1)).max()) < 2e-3 and cache.sync() == 0


@pytest.mark.parametrize("page,Hk,new,B", [(128, 1, 40, 152), (64, 4, 64, 38), (16, 2, 1, 60)])
def test_long_units_on_all_sms(P, page, Hk, new, B):
    cache = filled(P, torch.float16, B, Hk, page, 3000, seed=5)
    q = torch.randn(B * new, 2 * Hk, D, device=DEV).half()
    out = cache.attend(q, offsets_of([new] * B), new)
    check(cache, q, [new] * B, out, [3000] * B, only=(0, 7, B - 1))
    for _ in range(5):
        assert torch.equal(out, cache.attend(q, offsets_of([new] * B), new))
    assert cache.sync() == 0


@pytest.mark.parametrize("shared", [0, 2])
@pytest.mark.parametrize("max_new", [1, 30])
def test_no_new_tokens_at_all(P, shared, max_new):
    cache = filled(P, torch.bfloat16, 5, 2, 32, 100, shared=shared)
    before = cache.pages.clone()
    off = torch.zeros(6, dtype=torch.int32, device=DEV)
    x = torch.randn(7, 8, D, device=DEV).bfloat16()
    out = torch.full((7, 4, D), 3.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((7, 4, D), 3.0, dtype=torch.bfloat16, device=DEV)
    k, v = torch.full((7, 2, D), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((7, 2, D), 3.0, dtype=torch.bfloat16, device=DEV)
    cache.append(x[:, 4:6], x[:, 6:], off, q=x[:, :4], q_out=q)
    cache.attend(x[:, :4].contiguous(), off, max_new, shared_pages=shared, out=out)
    cache.read(off, 7, k_out=k, v_out=v)
    assert all(bool((t == 3).all()) for t in (out, q, k, v)) and torch.equal(cache.pages, before) and cache.sync() == 0
    assert cache.attend(x[:0, :4], off, 1).shape == (0, 4, D) and cache.read(off, 0)[0].shape == (0, 2, D)


@pytest.mark.parametrize("new", [1, 40])
def test_results_and_workspaces_are_memory_of_the_calls_stream(P, new):
    """Calls on a side stream, with outputs and workspaces made by the binding, while the current stream reuses memory."""
    cache = filled(P, torch.float16, 6, 2, 64, 900)
    q = torch.randn(6 * new, 8, D, device=DEV).half()
    off = offsets_of([new] * 6)
    want = cache.attend(q, off, new)
    k, v = cache.read(off, 6 * new)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = cache.attend(q, off, new, stream=side)
        rk, rv = cache.read(off, 6 * new, stream=side)
        junk = [torch.full((6 * new, 8, D), float("nan"), dtype=torch.float16, device=DEV) for _ in range(3)]
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(rk, k) and torch.equal(rv, v)
        del junk


def test_a_scores_jump_inside_a_tile(P):
    """Keys whose scores grow by far more than the weights' range inside one 128-key tile, in every half of it."""
    length, Hk = 700, 1
    for new in (1, 3, 40, 200):
        cache = filled(P, torch.float16, 1, Hk, 64, length, seed=9)
        g = torch.Generator(device=DEV).manual_seed(2)
        k = torch.randn(length, Hk, D, generator=g, device=DEV) * 0.01
        for at, size in ((0, 0.5), (20, 4.0), (70, 8.0), (130, 12.0), (200, 16.0), (300, 20.0), (470, 24.0), (650, 30.0)):
            k[at] = size
        v = torch.randn(length, Hk, D, generator=g, device=DEV)
        cache.append(k.half(), v.half(), offsets_of([length]))
        q = (0.2 + 0.01 * torch.randn(new, 4, D, generator=g, device=DEV)).half()
        out = cache.attend(q, offsets_of([new]), new)
        check(cache, q, [new], out, [length])
        q = -q                                                   # and one that falls
        check(cache, q, [new], cache.attend(q, offsets_of([new]), new), [length])
