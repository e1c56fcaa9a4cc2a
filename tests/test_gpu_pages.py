"""Pages planned on the device (include/pages.h): every array equals a plain
list-and-stack implementation's after every call; and rotation tables
(include/rope.h) against 64 bits.

Bar of the tables.  The reference's angles are exact to 2^-50 of themselves and
reduced before its cosine, so they cost nothing here; the kernel's value may be
off by 2^-22 of the magnitude (header).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


class Plain:
    """The rule of include/pages.h with lists."""

    def __init__(self, table, lengths, held, free, n_free, page):
        self.table, self.lengths, self.held = [list(map(int, r)) for r in table], list(map(int, lengths)), list(map(int, held))
        self.free, self.n_free, self.page, self.width = list(map(int, free)), int(n_free), page, len(table[0])

    def plan(self, new, tokens, shared=0):
        B = len(new)
        need, bad = [], 0
        for n, l, h in zip(new, self.lengths, self.held):
            if n < 0 or l < 0 or not 0 <= h <= self.width:
                bad |= 128
                need.append(h)
            elif l + n > self.width * self.page:
                bad |= 1
                need.append(h)
            else:
                need.append(max(-(-(l + n) // self.page), min(h, shared)))
        given = sum(max(h - n, 0) for h, n in zip(self.held, need))
        taken = sum(max(n - h, 0) for h, n in zip(self.held, need))
        if sum(max(n, 0) for n in new) > tokens or not 0 <= self.n_free <= len(self.free) or self.n_free + given > len(self.free):
            bad |= 128
        if taken > self.n_free + given:
            bad |= 1
        if bad:
            return [0] * (B + 1), [-1] * tokens, [-1] * tokens, bad
        for b in range(B):
            for j in range(need[b], self.held[b]):
                self.free[self.n_free] = self.table[b][j]
                self.n_free += 1
        for b in range(B):
            for j in range(self.held[b], need[b]):
                self.n_free -= 1
                self.table[b][j] = self.free[self.n_free]
            self.held[b] = need[b]
        offsets, positions, slots = [0], [], []
        for b in range(B):
            for t in range(self.lengths[b], self.lengths[b] + new[b]):
                positions.append(t)
                slots.append(self.table[b][t // self.page] * self.page + t % self.page)
            self.lengths[b] += new[b]
            offsets.append(offsets[-1] + new[b])
        pad = [-1] * (tokens - len(slots))
        return offsets, positions + pad, slots + pad, 0


def same(pool, plain, got, want):
    for g, w in zip(got, want[:3]):
        assert g.tolist() == w
    assert pool.page_table.tolist() == plain.table and pool.lengths.tolist() == plain.lengths
    assert pool.held.tolist() == plain.held and pool.free_pages.tolist() == plain.free and pool.n_free.item() == plain.n_free


def make(P, B, width, page, n_pages):
    table = torch.full((B, width), -7, dtype=torch.int32, device=DEV)
    lengths = torch.zeros(B, dtype=torch.int64, device=DEV)
    pool = P.PagePool(table, lengths, page, n_pages=n_pages)
    return pool, Plain(table.tolist(), lengths.tolist(), [0] * B, pool.free_pages.tolist(), n_pages, page)


@pytest.mark.parametrize("B,width,page,n_pages,most,tokens", [
    (1, 1, 1, 1, 1, 1), (1, 40, 16, 64, 70, 100), (3, 9, 16, 20, 20, 64), (33, 6, 64, 150, 9, 400), (511, 4, 7, 1500, 3, 2000),
    (513, 8, 32, 4000, 40, 30000), (4096, 3, 16, 9000, 2, 9000), (2, 3000, 16, 5000, 30000, 70000), (7, 50, 1, 300, 8, 60)])
def test_plans_follow_the_rule(P, B, width, page, n_pages, most, tokens):
    """Steps with growth, rollback to other lengths, sequences that end, refusals, padded rows."""
    rng = np.random.default_rng(B + width)
    pool, plain = make(P, B, width, page, n_pages)
    refused = 0
    for step in range(8):
        new = rng.integers(0, most + 1, B)
        if step % 3 == 2:                                          # back to shorter lengths first
            cut = [int(rng.integers(0, l + 1)) if rng.random() < 0.5 else l for l in plain.lengths]
            cut[0] = 0
            plain.lengths = cut
            pool.lengths.copy_(torch.tensor(cut))
        want = plain.plan([int(x) for x in new], tokens)
        got = pool.plan(torch.tensor(new, dtype=torch.int32, device=DEV), tokens)
        same(pool, plain, got, want)
        assert pool.error.item() == want[3]
        refused += want[3] != 0
        pool.error.zero_()
    pages = [p for b in range(B) for p in plain.table[b][:plain.held[b]]] + plain.free[:plain.n_free]
    assert sorted(pages) == list(range(n_pages)) and refused < 8


def test_shared_pages_are_kept(P):
    pool, plain = make(P, 3, 6, 16, 20)
    for b in range(3):
        plain.table[b][:2] = [17, 18]
    pool.page_table[:, :2] = torch.tensor([17, 18], dtype=torch.int32, device=DEV)
    plain.held, plain.lengths = [2, 2, 0], [32, 32, 0]
    pool.held.copy_(torch.tensor(plain.held))
    pool.lengths.copy_(torch.tensor(plain.lengths))
    for new, cut in (([5, 20, 40], None), ([1, 0, 3], [32, 33, 0]), ([0, 0, 0], [0, 5, 0])):
        if cut:
            plain.lengths = list(cut)
            pool.lengths.copy_(torch.tensor(cut))
        want = plain.plan(new, 80, shared=2)
        same(pool, plain, pool.plan(torch.tensor(new, dtype=torch.int32, device=DEV), 80, shared_pages=2), want)
    assert plain.held == [2, 2, 2] and pool.sync() == 0


@pytest.mark.parametrize("kind", ["pages", "table", "count", "length", "rows", "held", "free"])
def test_a_refused_call_changes_nothing(P, kind):
    pool, plain = make(P, 3, 4, 16, 8)
    new, tokens = [20, 3, 30], 64
    want = plain.plan(new, tokens)
    same(pool, plain, pool.plan(torch.tensor(new, dtype=torch.int32, device=DEV), tokens), want)
    new, bit = [1, 1, 1], 128
    if kind == "pages":
        new, bit = [40, 40, 30], 1 + 128                          # 110 tokens are also more than the 64 rows
    elif kind == "table":
        new, bit = [1, 62, 1], 1
    elif kind == "count":
        new = [1, -1, 1]
    elif kind == "length":
        plain.lengths[1] = -1
    elif kind == "rows":
        tokens = 2
    elif kind == "held":
        plain.held[0] = 5
    else:
        plain.n_free = 9
    pool.lengths.copy_(torch.tensor(plain.lengths))
    pool.held.copy_(torch.tensor(plain.held))
    pool.n_free.fill_(plain.n_free)
    want = plain.plan(new, tokens)
    got = pool.plan(torch.tensor(new, dtype=torch.int32, device=DEV), tokens)
    assert want[3] == bit and pool.error.item() == bit and got[0].tolist() == [0, 0, 0, 0]
    same(pool, plain, got, want)
    with pytest.raises(P.PaluError, match="device error word"):
        pool.sync()
    assert pool.sync() == 0


def test_a_captured_plan(P):
    pool, plain = make(P, 5, 8, 16, 30)
    new = torch.zeros(5, dtype=torch.int32, device=DEV)
    bufs = dict(offsets=torch.zeros(6, dtype=torch.int32, device=DEV), positions=torch.zeros(40, dtype=torch.int64, device=DEV),
                slots=torch.zeros(40, dtype=torch.int64, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.plan(new, 40, **bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.plan(new, 40, **bufs)
    for n in ([5, 0, 17, 1, 9], [1, 1, 1, 1, 1], [0, 30, 0, 0, 0], [8, 8, 8, 8, 8]):
        new.copy_(torch.tensor(n))
        graph.replay()
        torch.cuda.synchronize()
        same(pool, plain, (bufs["offsets"], bufs["positions"], bufs["slots"]), plain.plan(n, 40))
    assert pool.sync() == 0


def test_python_refusals(P):
    table, lengths = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    pool = P.PagePool(table, lengths, 16, n_pages=4)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: P.PagePool(table, lengths, 16), lambda: P.PagePool(table, lengths.int(), 16, n_pages=4),
                lambda: P.PagePool(table[0], lengths, 16, n_pages=4), lambda: P.PagePool(table, lengths, 16, held=new.long(), n_pages=4),
                lambda: P.PagePool(table, lengths, 16, free_pages=new), lambda: pool.plan(new.long(), 4),
                lambda: pool.plan(new[:1], 4), lambda: pool.plan(new, 4, slots=torch.zeros(3, dtype=torch.int64, device=DEV)),
                lambda: P.rope_table(4, 64, scaling="none"), lambda: P.rope_table(4, 64, out=torch.zeros(4, 32, device=DEV)),
                lambda: P.rope_table(4, 64, device="cpu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: P.PagePool(table, lengths, 0, n_pages=4), lambda: pool.plan(new, 4, shared_pages=5),
                lambda: P.PagePool(table, lengths, 16, held=table.view(-1)[:2], n_pages=4),
                lambda: pool.plan(pool.held, 4), lambda: P.rope_table(4, 24), lambda: P.rope_table(4, 64, base=1.0),
                lambda: P.rope_table(4, 64, scaling="linear", factor=0.5), lambda: P.rope_table(4, 64, scaling="parts", factor=2.0)):
        with pytest.raises(P.PaluError):
            bad()


# ------------------------------------------------------------------ rotation tables

def frequencies(d, base, scaling, factor, original, low, high):
    i = np.arange(0, d, 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (d / (d - 2))
    f = base ** (-i / d)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        t = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f * t + f / factor * (1 - t)
    return f


@pytest.mark.parametrize("n,d,start", [(1, 16, 0), (7, 128, 0), (1000, 64, 0), (333, 96, 100000), (5, 48, 1 << 40), (70001, 128, 0)])
@pytest.mark.parametrize("scaling,factor,base", [("plain", 1.0, 10000.0), ("linear", 4.0, 10000.0), ("ntk", 8.0, 10000.0),
                                                 ("parts", 16.0, 500000.0), ("parts", 1.0, 10000.0)])
def test_rope_table(P, n, d, start, scaling, factor, base):
    got = P.rope_table(n, d, base=base, scaling=scaling, factor=factor, original=8192, start=start).cpu().double()
    f = frequencies(d, base, scaling, factor, 8192, 1.0, 32.0)
    magnitude = 0.1 * math.log(factor) + 1 if scaling == "parts" else 1.0
    # position = far + near, each angle below 2^53 / 2^50 of a turn's error; far positions: the bar's angle term
    p = np.arange(start, start + n, dtype=np.float64)
    ang = p[:, None] * f
    ref = np.concatenate([np.cos(ang), np.sin(ang)], 1) * magnitude
    # both sides' angles are off by a few 2^-53 of the angle; 2^-50 of it covers the two
    slack = np.concatenate([ang, ang], 1) * 2.0 ** -50 + 2.0 ** -63 * (start + n) * 2 * math.pi
    err = np.abs(got.numpy() - ref)
    assert (err <= magnitude * (2.0 ** -22 + slack)).all(), float((err / magnitude).max())
    if start == 0:
        assert (got[0, :d // 2].numpy() == np.float32(magnitude)).all() and (got[0, d // 2:] == 0).all()


def test_rope_tables_feed_the_rotation(P):
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(1, 9, 2, 128, generator=g).to(DEV).half(), torch.randn(1, 9, 1, 128, generator=g).to(DEV).half()
    pos = torch.arange(9, device=DEV)[None]
    a = P.qk_norm_rope(q, k, pos + 50, P.rope_table(64, 128))
    b = P.qk_norm_rope(q, k, pos, P.rope_table(9, 128, start=50))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert P.rope_table(0, 64).shape == (0, 64)
