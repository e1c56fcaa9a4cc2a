"""The paged cache (include/paged.h) on the GPU against plain implementations
in 64 bits: norm and rotation of queries and keys, appends into pages, and
attention of new tokens over the pages with and without a shared prefix.

Bars.  Norm, rotation and append: fp32 arithmetic of a few operations (each
2^-24 relative, the norm's root and quotient a few of them; rotation adds two
products, so relative to the pair's length), then one rounding to the type
(at most eps / 2 of the value): |got - ref| <= (eps / 2 + 2^-19) * length of
the pair.  Attention: the output is a weighted mean of value rows.  The
weights are rounded to the type once (eps / 2 each, the kernels for many rows) and
the output once more; scores carry 128 fp32-accumulated products of inputs of
size a few, about 2^-16 absolute, which enters every weight relatively.  So
with A = sum of weights * |v| (computed per output in 64 bits):
|got - ref| <= (eps / 2 + 2^-12) * A + (eps / 2) * |ref|.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
D = 128
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


def _table(n_pos, rope):
    half = rope // 2
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def ref_transform(x, w, cs, interleaved, eps):
    """x [..., H, 128] (any type), cs [..., rope] or None: fp64 result and the length of each channel's pair."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    scale = x.abs().clone()
    if cs is not None:
        rope = cs.shape[-1]
        n = torch.arange(rope // 2)
        i, j = (2 * n, 2 * n + 1) if interleaved else (n, n + rope // 2)
        c, s = cs[..., None, :rope // 2].double(), cs[..., None, rope // 2:].double()
        a, b = x[..., i].clone(), x[..., j].clone()
        x[..., i] = a * c - b * s
        x[..., j] = b * c + a * s
        scale[..., i] = scale[..., j] = (a * a + b * b).sqrt()
    return x, scale


def close(got, ref, scale, dt):
    eps = torch.finfo(dt).eps
    tiny = torch.finfo(dt).smallest_normal * eps      # half a step among the subnormals
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= (eps / 2 + 2.0 ** -19) * scale + tiny).all()), float((err / (scale + tiny)).max())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,rope,inter,norm", [
    (1, 1, 1, 1, 128, False, True), (3, 5, 7, 1, 64, True, True), (2, 33, 24, 8, 32, False, False),
    (1, 257, 28, 4, 128, True, True), (5, 3, 5, 5, 96, False, True), (2, 17, 9, 3, 16, True, False),
    (2, 4, 4, 2, 0, False, True), (1, 6, 4, 4, 0, False, False), (1, 3, 6, 2, 112, True, True)])
def test_norm_and_rotation(P, dt, B, T, Hq, Hk, rope, inter, norm):
    g = torch.Generator().manual_seed(B * 1000 + T)
    d = DT[dt]
    # views of one projection, with a gap between tokens
    qkv = torch.randn(B, T + 2, Hq + 2 * Hk + 1, D, generator=g).to(d)
    qkv[0, 0, 0] *= 40
    q, k = qkv[:, 1:T + 1, :Hq], qkv[:, 1:T + 1, Hq:Hq + Hk]
    pos = torch.randint(0, 5000, (B, T), generator=g)
    cs = _table(5000, rope) if rope else None
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(d) if norm else None for _ in range(2)]
    dev = lambda t: None if t is None else t.to(DEV)
    qkvd = qkv.to(DEV)
    qo, ko = P.qk_norm_rope(qkvd[:, 1:T + 1, :Hq], qkvd[:, 1:T + 1, Hq:Hq + Hk], dev(pos), dev(cs), dev(w[0]), dev(w[1]),
                            eps=1e-5, interleaved=inter)
    for got, x, ww in ((qo, q, w[0]), (ko, k, w[1])):
        ref, scale = ref_transform(x, ww, None if cs is None else cs[pos], inter, 1e-5)
        assert got.shape == (B, x.shape[2], T, D) and got.is_contiguous()
        close(got, ref.transpose(1, 2), scale.transpose(1, 2), d)


def test_norm_of_one_operand_zero_rows_and_large_values(P):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 2, 3, D, generator=g).half()
    q[0, 0, 1] = 0
    q[0, 1, 2] = 60000.0                                       # squares beyond fp16, a sum within fp32
    k = torch.randn(1, 2, 1, D, generator=g).half()
    w = torch.ones(D).half()
    qo, ko = P.qk_norm_rope(q.to(DEV), k.to(DEV), None, None, q_weight=w.to(DEV), eps=1e-6)
    ref, scale = ref_transform(q, w, None, False, 1e-6)
    close(qo, ref.transpose(1, 2), scale.transpose(1, 2), torch.float16)
    assert torch.equal(ko.cpu(), k.transpose(1, 2))            # neither norm nor rotation: the bits


def test_position_outside_the_table(P):
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(2, 2, 4, D, generator=g).half().to(DEV), torch.randn(2, 2, 2, D, generator=g).half().to(DEV)
    pos = torch.tensor([[0, 9], [10, -1]], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, ko = P.qk_norm_rope(q, k, pos, _table(10, 64).to(DEV), error=err)
    assert err.item() == P.PALU_DEVERR_POSITION
    assert torch.isnan(qo[1]).all() and torch.isnan(ko[1]).all()
    assert torch.isfinite(qo[0]).all() and torch.isfinite(ko[0]).all()


# ------------------------------------------------------------------ paged

def make_cache(P, dt, lengths, page, Hk, layout="heads", spare=2, seed=0, fill=None, shared=0, width=None):
    """Pools (host copy and device view), a page table without order, the cache.  fill: what unwritten rows hold."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    width = width or max(1, -(-max(max(lengths), 1) // page))
    n_pages = B * width + spare
    ids = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).to(torch.int32)
    ids[:, :shared] = ids[0, :shared]
    pools = []
    for _ in range(2):
        x = torch.randn(n_pages, Hk, page, D, generator=g) + 0.5 * torch.randn(Hk, 1, D, generator=g)
        pools.append(x.to(dt))
    if fill is not None:
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for t in range(n):
                used[ids[b, t // page], t % page] = True
        for x in pools:
            x.transpose(1, 2)[~used] = fill
    if layout == "heads":
        dev = [x.to(DEV) for x in pools]
    elif layout == "tokens":
        dev = [x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for x in pools]
    else:  # keys and values of a page beside each other, heads padded by one
        both = torch.zeros(n_pages, 2, Hk + 1, page, D, dtype=dt)
        both[:, 0, :Hk], both[:, 1, :Hk] = pools
        both = both.to(DEV)
        dev = [both[:, 0, :Hk], both[:, 1, :Hk]]
    table, length = ids.to(DEV), torch.tensor(lengths, dtype=torch.int64, device=DEV)
    return pools, dev, P.PagedCache(dev[0], dev[1], table, length)


def offsets_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("layout", ["heads", "tokens", "pairs"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,rope,inter", [
    (16, [1], [1], 4, 4, 128, False), (16, [3, 0, 17, 1], [3, 40, 33, 100], 7, 1, 64, True),
    (64, [1] * 5, [1, 64, 65, 128, 500], 28, 4, 128, False), (128, [200, 5], [200, 300], 6, 3, 32, True)])
def test_append(P, dt, layout, page, new, lengths, Hq, Hk, rope, inter):
    d = DT[dt]
    g = torch.Generator().manual_seed(sum(new) + page)
    pools, dev, c = make_cache(P, d, lengths, page, Hk, layout)
    n, pad = sum(new), 3
    qkv = torch.randn(n + pad, Hq + 2 * Hk, D, generator=g).to(d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    cs = _table(max(lengths), rope)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(d) for _ in range(2)]
    qkvd = qkv.to(DEV)
    q_out = torch.full((n + pad, Hq, D), 7.0, dtype=d, device=DEV)
    r = c.append(qkvd[:, Hq:Hq + Hk], qkvd[:, Hq + Hk:], offsets_of(new), q=qkvd[:, :Hq], cos_sin=cs.to(DEV),
                 q_weight=w[0].to(DEV), k_weight=w[1].to(DEV), interleaved=inter, q_out=q_out)
    assert r is q_out and c.sync() == 0
    assert (q_out[n:] == 7).all()                                   # padded rows
    ids, row = c.page_table.cpu(), 0
    kref, vref = pools[0].clone().double(), pools[1].clone()
    kscale = torch.zeros_like(kref)
    kscale[:] = kref.abs()
    for b, m in enumerate(new):
        pos = torch.arange(lengths[b] - m, lengths[b])
        sl = slice(row, row + m)
        ref, scale = ref_transform(q[sl], w[0], cs[pos], inter, 1e-6)
        close(q_out[sl], ref, scale, d)
        ref, scale = ref_transform(k[sl], w[1], cs[pos], inter, 1e-6)
        at = ids[b].long()[pos // page], slice(None), pos % page
        kref[at], kscale[at], vref[at] = ref, scale, v[sl]
        row += m
    close(dev[0], kref, kscale, d)                                  # every other row as it was
    assert torch.equal(dev[1].cpu(), vref)


def test_append_without_queries_or_transform_copies(P):
    lengths, new = [5, 20], [5, 4]
    pools, dev, c = make_cache(P, torch.float16, lengths, 16, 2)
    k, v = torch.randn(2, 9, 2, D).half().to(DEV)
    assert c.append(k, v, offsets_of(new)) is None
    ids = c.page_table.cpu().long()
    for x, y, pool in ((k, dev[0], pools[0]), (v, dev[1], pools[1])):
        want = pool.clone()
        want[ids[0, 0], :, :5] = x[:5].cpu().transpose(0, 1)
        for i in range(4):
            want[ids[1, (16 + i) // 16], :, (16 + i) % 16] = x[5 + i].cpu()
        assert torch.equal(y.cpu(), want)


def test_append_refused_on_the_device(P):
    """Each refusal: its bit, NaN queries, nothing written, the other sequences served."""
    for bit, break_it in (
            (P.PALU_DEVERR_CAPACITY, lambda c: c.lengths.__setitem__(1, 33)),
            (P.PALU_DEVERR_SPAN, lambda c: c.lengths.__setitem__(1, 1)),
            (P.PALU_DEVERR_PAGE, lambda c: c.page_table.__setitem__((1, 1), 99)),
            (P.PALU_DEVERR_PAGE, lambda c: c.page_table.__setitem__((1, 1), -1)),
            (P.PALU_DEVERR_POSITION, None)):
        pools, dev, c = make_cache(P, torch.bfloat16, [4, 30, 9], 16, 2, width=2)
        k, v = torch.randn(2, 6, 2, D).bfloat16().to(DEV)
        q = torch.randn(6, 4, D).bfloat16().to(DEV)
        if break_it:
            break_it(c)
        cs = _table(40 if break_it else 20, 128).to(DEV)
        qo = c.append(k, v, offsets_of([2, 2, 2]), q=q, cos_sin=cs)
        with pytest.raises(P.PaluError) as e:
            c.sync()
        assert e.value.status == 6 and f"word {bit}:" in str(e.value)
        assert c.sync() == 0
        assert torch.isnan(qo[2:4]).all() and torch.isfinite(qo[:2]).all() and torch.isfinite(qo[4:]).all()
        ids = c.page_table.cpu().long()
        want = pools[1].clone()
        for t, p in ((0, 2), (1, 3)):
            want[ids[0, 0], :, p] = v[t].cpu()
        for t, p in ((4, 7), (5, 8)):
            want[ids[2, 0], :, p] = v[t].cpu()
        assert torch.equal(dev[1].cpu(), want)


def ref_attend(q, pools, ids, lengths, new, page, scale=None):
    """fp64 attention and, per output, the weighted sum of |v|."""
    Hq, Hk = q.shape[1], pools[0].shape[1]
    G = Hq // Hk
    out, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            lim = lengths[b] - n + i + 1
            if lim > 0:
                t = torch.arange(lim)
                at = ids[b].long()[t // page], slice(None), t % page
                k = pools[0][at].double().repeat_interleave(G, 1)   # [lim, Hq, D]
                v = pools[1][at].double().repeat_interleave(G, 1)
                s = torch.einsum("hd,thd->ht", q[row].double(), k) * (scale or 1 / math.sqrt(D))
                p = torch.softmax(s, -1)
                out[row] = torch.einsum("ht,thd->hd", p, v)
                mag[row] = torch.einsum("ht,thd->hd", p, v.abs())
            row += 1
    return out, mag


def attend_close(got, ref, mag, dt):
    eps = torch.finfo(dt).eps
    err = (got.cpu().double() - ref).abs()
    bar = (eps / 2 + 2.0 ** -12) * mag + eps / 2 * ref.abs() + torch.finfo(dt).smallest_normal * eps
    assert torch.isfinite(got).all()
    assert bool((err <= bar).all()), float((err / bar).max())


CASES = [  # page, new, lengths, Hq, Hk, shared pages
    (16, [1], [1], 1, 1, 0), (16, [1], [2], 3, 1, 0), (32, [1], [513], 24, 8, 0), (64, [1, 1, 1], [127, 128, 129], 7, 1, 0),
    (16, [1, 0, 1, 1], [300, 77, 1, 16], 8, 2, 0), (128, [1] * 6, [5000, 17, 333, 1024, 1, 129], 28, 4, 0),
    (16, [5, 2, 0, 3], [5, 200, 9, 131], 6, 3, 0), (32, [2, 2], [2, 500], 16, 2, 0),
    (64, [40, 1, 13], [40, 700, 260], 12, 4, 0), (16, [130], [130], 8, 1, 0), (128, [300, 77], [300, 1000], 10, 2, 0),
    (16, [1, 1, 1], [40, 33, 50], 3, 1, 2), (32, [1] * 9, [300 + 31 * i for i in range(9)], 24, 8, 9),
    (64, [5, 1, 4, 0, 5], [700, 641, 1000, 650, 645], 28, 4, 10), (128, [3] * 30, [515 + i for i in range(30)], 14, 2, 4),
    (16, [20, 7, 1], [1000, 800, 780], 16, 2, 47), (64, [1] * 40, [64 * 20 + 1 + 3 * i for i in range(40)], 8, 1, 20),
    (16, [1, 1], [4096, 4097], 40, 1, 256), (32, [70, 70, 70], [200, 150, 333], 64, 1, 2),
]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,shared", CASES)
def test_attend(P, dt, page, new, lengths, Hq, Hk, shared):
    d = DT[dt]
    layout = ("heads", "tokens", "pairs")[len(lengths) % 3]
    # what lies behind a sequence's length must not matter
    pools, dev, c = make_cache(P, d, lengths, page, Hk, layout, seed=page + Hq, fill=float("nan"), shared=shared)
    g = torch.Generator().manual_seed(len(new) + Hk)
    n, pad = sum(new), 2
    q = torch.randn(n + pad, Hq + 1, D, generator=g).to(d)
    out = torch.full((n + pad, Hq, D), 7.0, dtype=d, device=DEV)
    got = c.attend(q.to(DEV)[:, :Hq], offsets_of(new), max(new), shared_pages=shared, out=out)
    assert got is out and c.sync() == 0
    assert (out[n:] == 7).all()
    ref, mag = ref_attend(q[:n, :Hq], pools, c.page_table.cpu(), lengths, new, page)
    attend_close(out[:n], ref, mag, d)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("shared", [0, 3])
def test_rows_that_see_nothing_are_zero(P, dt, shared):
    """Lengths of zero, of less than the new tokens, and less than the shared prefix."""
    lengths, new = [0, 2, 70, 30], [1, 4, 1, 3]
    pools, dev, c = make_cache(P, DT[dt], lengths, 16, 2, seed=5, width=5, shared=shared)
    q = torch.randn(9, 8, D, generator=torch.Generator().manual_seed(1)).to(DT[dt])
    out = c.attend(q.to(DEV), offsets_of(new), 4, shared_pages=shared)
    assert c.sync() == 0
    ref, mag = ref_attend(q, pools, c.page_table.cpu(), lengths, new, 16)
    assert (out[:3] == 0).all() and (ref[:3] == 0).all()
    attend_close(out, ref, mag, DT[dt])


@pytest.mark.parametrize("Hq,Hk,new", [(4, 2, 1), (6, 1, 3)])
def test_many_short_sequences(P, Hq, Hk, new):
    """A thousand sequences, many without new tokens, some empty: more than a CTA's threads."""
    rng = np.random.default_rng(new)
    B = 1000
    counts = [int(rng.integers(0, new + 1)) for _ in range(B)]
    lengths = [max(int(rng.integers(0, 60)), n) for n in counts]
    pools, dev, c = make_cache(P, torch.float16, lengths, 16, Hk, seed=8, width=4)
    n = sum(counts)
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(7)).half()
    out = c.attend(q.to(DEV), offsets_of(counts), new)
    assert c.sync() == 0
    ref, mag = ref_attend(q, pools, c.page_table.cpu(), lengths, counts, 16)
    attend_close(out, ref, mag, torch.float16)
    k, v = torch.randn(2, n, Hk, D, generator=torch.Generator().manual_seed(9)).half()
    c.append(k.to(DEV), v.to(DEV), offsets_of(counts))
    ids, row = c.page_table.cpu().long(), 0
    for b, m in enumerate(counts):
        for t in range(lengths[b] - m, lengths[b]):
            pools[0][ids[b, t // 16], :, t % 16], pools[1][ids[b, t // 16], :, t % 16] = k[row], v[row]
            row += 1
    assert torch.equal(dev[0].cpu(), pools[0]) and torch.equal(dev[1].cpu(), pools[1])


def test_no_new_tokens_at_all(P):
    """Offsets of zero throughout: padded rows only, nothing is touched."""
    for shared in (0, 2):
        pools, dev, c = make_cache(P, torch.bfloat16, [40, 0, 33], 16, 2, width=3, shared=shared)
        off = torch.zeros(4, dtype=torch.int32, device=DEV)
        for n, mx in ((3, 1), (40, 40)):
            q = torch.zeros(n, 8, D, dtype=torch.bfloat16, device=DEV)
            out = torch.full((n, 8, D), 7.0, dtype=torch.bfloat16, device=DEV)
            c.attend(q, off, mx, shared_pages=shared, out=out)
            c.append(q[:, :2], q[:, 2:4], off)
            assert (out == 7).all() and c.sync() == 0
        assert torch.equal(dev[0].cpu(), pools[0])


def test_large_scores_scale_and_flat_rows(P):
    lengths, new = [400, 250], [1, 12]
    pools, dev, c = make_cache(P, torch.float16, lengths, 32, 2, seed=9)
    q = torch.randn(13, 4, D, generator=torch.Generator().manual_seed(2)).half()
    q[0, 0] = 0                                                     # flat: the mean of the values
    for scale in (0.0, 1e-3, 1.0):                                  # at 1.0 one token takes nearly all
        out = c.attend(q.to(DEV), offsets_of(new), 12, softmax_scale=scale)
        ref, mag = ref_attend(q, pools, c.page_table.cpu(), lengths, new, 32, scale or None)
        eps = torch.finfo(torch.float16).eps
        # scores of size 12 / scale of 1: 2^-24 * 128 products of size up to 4 sqrt(128) each enter the weights
        tol = (eps / 2 + 2.0 ** -12 + (2.0 ** -11 if scale == 1.0 else 0)) * mag + eps / 2 * ref.abs() + 2.0 ** -24
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_one_large_weight_among_many_small_ones(P, dt):
    """A first token whose weight is 2^14 .. 2^21 times every other's, of which there are 20,000: their sum counts."""
    S, new = 20000, 20
    pools, dev, c = make_cache(P, DT[dt], [S], 64, 1, seed=12)
    ids = c.page_table.cpu().long()
    q = torch.full((new, 2, D), 0.25).to(DT[dt])
    k = torch.zeros(S, D)
    k[0] = 44.0                                            # score 128 * 0.25 * 44 / sqrt(128) = 124.5, the others' 110 .. 114.6
    k[1:] = torch.linspace(38.9, 40.5, S - 1)[torch.randperm(S - 1, generator=torch.Generator().manual_seed(1))][:, None]
    pools[0][ids[0, torch.arange(S) // 64], 0, torch.arange(S) % 64] = k.to(DT[dt])
    dev[0].copy_(pools[0])
    for n in (1, new):
        out = c.attend(q[:n].to(DEV), offsets_of([n]), n)
        ref, mag = ref_attend(q[:n], pools, ids, [S], [n], 64)
        eps = torch.finfo(DT[dt]).eps
        # scores of 124 with 128 products of size 11: fp32 sums are right to about 128 * 124 * 2^-24 = 2^-10 at worst
        bar = (eps / 2 + 2.0 ** -9) * mag + eps / 2 * ref.abs()
        assert bool(((out.cpu().double() - ref).abs() <= bar).all())


def test_attend_refused_on_the_device(P):
    def fresh():
        return make_cache(P, torch.float16, [40, 33], 16, 2, seed=11, width=3)
    q = torch.randn(3, 4, D, generator=torch.Generator().manual_seed(3)).half()
    pools, dev, c = fresh()
    good, mag = ref_attend(q, pools, c.page_table.cpu(), [40, 33], [1, 2], 16)

    def word(c):
        with pytest.raises(P.PaluError) as e:
            c.sync()
        return int(str(e.value).split("word ")[1].split(":")[0])
    for shared in (0, 1):
        # more rows than max_new, offsets out of order: zeros for that sequence, the other one served
        pools, dev, c = fresh()
        out = c.attend(q.to(DEV), offsets_of([1, 2]), 1, shared_pages=0)
        assert word(c) == P.PALU_DEVERR_SPAN and (out[1:] == 0).all()
        attend_close(out[:1], good[:1], mag[:1], torch.float16)
        out = c.attend(q.to(DEV), torch.tensor([0, 1, 9], dtype=torch.int32, device=DEV), 2)
        assert word(c) == P.PALU_DEVERR_SPAN and (out[1:] == 0).all()
        # a page outside the pool: an error, no fault
        pools, dev, c = fresh()
        c.page_table[1, 1] = 1 << 20
        out = c.attend(q.to(DEV), offsets_of([1, 2]), 2)
        assert word(c) == P.PALU_DEVERR_PAGE
        attend_close(out[:1], good[:1], mag[:1], torch.float16)
        # a length past the table is cut to it
        pools, dev, c = fresh()
        c.lengths[1] = 1000
        c.attend(q.to(DEV), offsets_of([1, 2]), 2)
        assert word(c) == P.PALU_DEVERR_CAPACITY


@pytest.mark.parametrize("shared", [0, 1])
def test_rows_before_the_first_sequence_and_bad_spans(P, shared):
    """Offsets that begin behind 0, or that a sequence has too many rows of: the error word and zeros, with a shared prefix
    or without, and the other sequences served."""
    q = torch.randn(9, 4, D, generator=torch.Generator().manual_seed(3)).half()
    for first, new, max_new, bad in ((2, [1, 2, 1], 2, []), (7, [1, 0, 1], 40, []), (0, [1, 7, 1], 6, [1]), (0, [6, 1, 2], 2, [0]),
                                     (3, [0, 0, 0], 2, [])):
        lengths = [40, 33, 25]
        pools, dev, c = make_cache(P, torch.float16, lengths, 16, 2, seed=11, width=3, shared=shared)
        out = torch.full((9, 4, D), 7.0, dtype=torch.float16, device=DEV)
        off = offsets_of(new) + first
        end = first + sum(new)
        c.attend(q.to(DEV), off, max_new, shared_pages=shared, out=out)
        with pytest.raises(P.PaluError) as e:
            c.sync()
        assert f"word {P.PALU_DEVERR_SPAN}:" in str(e.value)
        assert (out[end:] == 7).all() and (out[:first] == 0).all()
        ref, mag = ref_attend(q[first:end], pools, c.page_table.cpu(), lengths, new, 16)
        row = 0
        for b, n in enumerate(new):
            if b in bad:
                assert (out[first + row:first + row + n] == 0).all()
            elif n:
                attend_close(out[first + row:first + row + n], ref[row:row + n], mag[row:row + n], torch.float16)
            row += n


@pytest.mark.parametrize("n", [1, 3000])
def test_all_rows_of_a_large_call_see_nothing(P, n):
    pools, dev, c = make_cache(P, torch.bfloat16, [0, 0], 16, 2, seed=3, width=5)
    q = torch.randn(2 * n, 64, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    out = torch.full((2 * n + 1, 64, D), 7.0, dtype=torch.bfloat16, device=DEV)
    c.attend(q, offsets_of([n, n]), n, out=out[:-1])
    assert c.sync() == 0 and (out[:-1] == 0).all() and (out[-1] == 7).all()


def test_shared_prefix_does_not_change_the_result(P):
    lengths, new, page, shared = [1000, 900, 1100], [4, 4, 4], 64, 13
    pools, dev, c = make_cache(P, torch.bfloat16, lengths, page, 4, seed=21, shared=shared)
    q = torch.randn(12, 16, D, generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    ref, mag = ref_attend(q.cpu(), pools, c.page_table.cpu(), lengths, new, page)
    for s in range(0, shared + 1, 3):
        attend_close(c.attend(q, offsets_of(new), 4, shared_pages=s), ref, mag, torch.bfloat16)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("Hk,new", [(1, 5), (2, 40)])
def test_long_units_on_all_sms(P, page, Hk, new):
    """More sequences than SMs, each long: the tiles of a unit of up to 128 rows go to two independent halves, those of
    a larger one to both.  Compared with the same tokens attended one at a time (another kernel); A of the bar is
    the same attention over |v|."""
    B, G, S = 160, 8 // Hk if new == 5 else 4, 4096 + 100
    g = torch.Generator(device=DEV).manual_seed(page + new)
    width = -(-S // page)
    ids = torch.randperm(B * width, generator=g, device=DEV).view(B, width).to(torch.int32)
    k, v = (torch.randn(B * width, Hk, page, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    lengths = S - torch.arange(B, device=DEV, dtype=torch.int64) * 7 % 1000
    c = P.PagedCache(k, v, ids, lengths)
    q = torch.randn(B, new, Hk * G, D, generator=g, device=DEV).bfloat16()
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    out = [c.attend(q.view(B * new, Hk * G, D), off * new, new).view(q.shape) for _ in range(3)]
    assert c.sync() == 0 and torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    eps = torch.finfo(torch.bfloat16).eps
    for i in sorted({0, 1, new // 2, new - 1}):
        at = lengths - (new - 1 - i)
        one = P.PagedCache(k, v, ids, at).attend(q[:, i].contiguous(), off, 1).float()
        mag = P.PagedCache(k, v.abs(), ids, at).attend(q[:, i].contiguous(), off, 1).float()
        bar = (eps / 2 + 2.0 ** -12) * mag * (1 + eps) + eps * one.abs() * (1 + eps)   # two roundings of the output
        assert bool(((out[0][:, i].float() - one).abs() <= bar).all())


SHARED = [  # page, new, lengths, Hq, Hk, shared pages: sizes at which the shared pages are read once
    (16, [1] * 8, [257 + 40 * i for i in range(8)], 64, 64, 16), (64, [1] * 8, [257, 300, 256, 700, 0, 1, 255, 600], 64, 64, 4),
    (16, [1] * 8, [288 + 37 * i for i in range(8)], 128, 64, 17), (128, [1] * 30, [257 + 60 * i for i in range(30)], 64, 32, 2),
    (32, [2, 0, 1, 2, 2, 1, 0, 2], [700, 300, 290, 258, 257, 256, 20, 500], 64, 64, 8),
    (16, [1, 5, 3, 5, 0, 5, 2, 4], [560, 516, 900, 512, 300, 570, 257, 515], 128, 64, 32),
    (64, [20, 20, 1, 7, 20, 3, 0, 20], [700, 532, 600, 515, 300, 513, 10, 560], 96, 96, 8),
    (32, [9, 1, 1, 9, 1, 2, 1, 1], [700, 641, 640, 649, 100, 660, 680, 661], 128, 32, 20),
    (32, [1] * 6, [400, 256, 257, 290, 10, 500], 96, 96, 8),
    (128, [3] * 30, [257 + 2 * i for i in range(30)], 48, 48, 2),
]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,shared", SHARED)
def test_shared_pages_are_read_once(P, dt, page, new, lengths, Hq, Hk, shared):
    """The other sequences' leading table entries name a page of NaN in the second call: only row 0's are read."""
    d = DT[dt]
    pools, dev, c = make_cache(P, d, lengths, page, Hk, seed=page + sum(lengths), shared=shared, spare=2)
    n = sum(new)
    q = torch.randn(n + 2, Hq, D, generator=torch.Generator().manual_seed(n)).to(d)
    ref, mag = ref_attend(q[:n], pools, c.page_table.cpu(), lengths, new, page)
    ws = c.attend_workspace(n + 2, Hq, max(new), shared)
    out = [torch.full((n + 2, Hq, D), 7.0, dtype=d, device=DEV) for _ in range(3)]
    c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared, workspace=ws, out=out[0])
    c.attend(q.to(DEV), offsets_of(new), max(new), workspace=ws, out=out[1])
    free = sorted(set(range(dev[0].shape[0])) - set(c.page_table.flatten().tolist()))[0]
    for t in dev:
        t[free] = float("nan")
    c.page_table[1:, :shared] = free
    c.attend(q.to(DEV), offsets_of(new), max(new), shared_pages=shared, workspace=ws, out=out[2])
    assert c.sync() == 0
    for o in out:
        assert (o[n:] == 7).all()
        attend_close(o[:n], ref, mag, d)
    assert torch.equal(out[0], out[2])


@pytest.mark.parametrize("new,shared", [([600, 1, 300, 0], 3), ([1500, 1500, 2, 1], 20)])
def test_long_chunks_with_a_shared_prefix(P, new, shared):
    """Chunks of many row tiles with shared pages named, against the same call without: spot rows against 64 bits."""
    page, Hq, Hk = 64, 28, 4
    lengths = [page * shared + n + 5 for n in new]
    pools, dev, c = make_cache(P, torch.bfloat16, lengths, page, Hk, seed=41, shared=shared)
    n = sum(new)
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    off = offsets_of(new)
    a = c.attend(q.to(DEV), off, max(new), shared_pages=shared)
    b = c.attend(q.to(DEV), off, max(new))
    assert c.sync() == 0
    eps = torch.finfo(torch.bfloat16).eps
    row = 0
    for i, m in enumerate(new):
        for t in sorted({0, m // 3, m - 1}) if m else ():
            ref, mag = ref_attend(q[row + t:row + t + 1], pools, c.page_table.cpu()[i:i + 1], [lengths[i] - (m - 1 - t)], [1], page)
            for o in (a, b):
                attend_close(o[row + t:row + t + 1], ref, mag, torch.bfloat16)
        row += m
    # all rows: both lie within the bar of the exact value, whose size is bounded by the largest value
    top = max(float(x.abs().max()) for x in pools[1:])
    assert float((a.float() - b.float()).abs().max()) <= 2 * (eps + 2.0 ** -12) * top


def test_calls_repeat_bit_for_bit(P):
    pools, dev, c = make_cache(P, torch.float16, [3000, 17, 900], 32, 4, seed=22, shared=0)
    q = torch.randn(15, 12, D, generator=torch.Generator().manual_seed(5)).half().to(DEV)
    for new in ([1, 1, 1], [5, 5, 5]):
        a = c.attend(q[:sum(new)], offsets_of(new), max(new))
        for _ in range(3):
            assert torch.equal(a, c.attend(q[:sum(new)], offsets_of(new), max(new)))


def test_offsets_beyond_32_bits_in_a_large_pool(P):
    """Pages whose element offset passes 2^31: the last pages of a 10 GB pool."""
    page, Hk = 128, 8
    n_pages = (1 << 32) // (page * Hk * D) + 40
    pool = torch.zeros(2, n_pages, Hk, page, D, dtype=torch.float16, device=DEV)
    ids = torch.tensor([[n_pages - 1, 3, n_pages - 7]], dtype=torch.int32, device=DEV)
    length = torch.tensor([300], dtype=torch.int64, device=DEV)
    c = P.PagedCache(pool[0], pool[1], ids, length)
    g = torch.Generator().manual_seed(6)
    k, v = torch.randn(2, 300, Hk, D, generator=g).half()
    q = torch.randn(300, 8, D, generator=g).half()
    c.append(k.to(DEV), v.to(DEV), offsets_of([300]))
    assert torch.equal(pool[0, n_pages - 1, :, 5].cpu(), k[5]) and torch.equal(pool[1, n_pages - 7, :, 43].cpu(), v[299])
    small = [torch.zeros(3, Hk, page, D, dtype=torch.float16) for _ in range(2)]
    for x, y in zip(small, (k, v)):
        for t in range(300):
            x[t // page, :, t % page] = y[t]
    for new in (1, 20):
        out = c.attend(q[-new:].to(DEV), offsets_of([new]), new)
        ref, mag = ref_attend(q[-new:], small, torch.arange(3)[None], [300], [new], page)
        attend_close(out, ref, mag, torch.float16)


def test_captured_graph_follows_lengths_and_pages(P):
    """A captured append and attention, replayed after the program changed lengths, table, offsets and inputs."""
    page, Hq, Hk, B = 32, 8, 2, 3
    pools, dev, c = make_cache(P, torch.float16, [100, 100, 100], page, Hk, seed=30, width=6)
    k, v = torch.randn(2, 6, Hk, D).half().to(DEV)
    q = torch.randn(6, Hq, D).half().to(DEV)
    cs = _table(200, 128).to(DEV)
    off = offsets_of([2, 2, 2])
    ws = c.attend_workspace(6, Hq, 2)
    out = torch.zeros(6, Hq, D, dtype=torch.float16, device=DEV)
    q_out = torch.zeros_like(out)

    def step():
        c.append(k, v, off, q=q, cos_sin=cs, q_out=q_out)
        c.attend(q_out, off, 2, workspace=ws, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(8)
    for lengths, new in (([101, 64, 180], [2, 1, 2]), ([3, 150, 33], [0, 2, 1])):
        c.lengths.copy_(torch.tensor(lengths))
        off.copy_(offsets_of(new))
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).half())
        graph.replay()
        torch.cuda.synchronize()
        assert c.sync() == 0
        n = sum(new)
        ref, mag = ref_attend(q_out[:n].cpu(), [d.cpu() for d in dev], c.page_table.cpu(), lengths, new, page)
        attend_close(out[:n], ref, mag, torch.float16)


@pytest.mark.parametrize("shared,new", [(0, 2), (3, 1), (3, 6)])
def test_copies_and_fills_between_the_calls(P, shared, new):
    """Inputs copied and outputs filled right before the calls and results read right behind them, eagerly and in a
    captured graph: the launches begin early, but never before the work ahead of them has ended."""
    page, Hq, Hk, B = 32, 8, 2, 40
    lengths = [page * shared + 40 + 7 * i for i in range(B)]
    pools, dev, c = make_cache(P, torch.bfloat16, lengths, page, Hk, seed=33, shared=shared, width=shared + 11)
    g = torch.Generator().manual_seed(10)
    n = B * new
    src = torch.randn(4, n, Hq + 2 * Hk, D, generator=g).bfloat16().to(DEV)
    x, off = torch.empty_like(src[0]), offsets_of([new] * B)
    cs = _table(1000, 128).to(DEV)
    ws = c.attend_workspace(n, Hq, new, shared)
    q, out, res = (torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    pick = torch.zeros(1, dtype=torch.int64, device=DEV)
    base = torch.tensor(lengths, device=DEV)
    grow = torch.zeros(1, dtype=torch.int64, device=DEV)

    def step():
        x.copy_(src[pick][0])                     # a kernel
        c.lengths.copy_(base)                     # a copy
        c.lengths.add_(grow)
        q.zero_()                                 # a fill
        c.append(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], off, q=x[:, :Hq], cos_sin=cs, q_out=q)
        out.zero_()
        c.attend(q, off, new, shared_pages=shared, workspace=ws, out=out)
        res.copy_(out)
        c.attend(q, off, new, shared_pages=shared, workspace=ws, out=out)

    def check(i):
        pick.fill_(i)
        grow.fill_(i)
        run()
        a, b = res.clone(), out.clone()
        assert torch.equal(a, b) and c.sync() == 0
        host, at = [t.cpu() for t in dev], [v + i for v in lengths]
        rows = torch.cat([torch.arange(b * new, (b + 1) * new) for b in (0, 17, B - 1)])
        ref, mag = ref_attend(q[rows].cpu(), host, c.page_table.cpu()[[0, 17, B - 1]], [at[0], at[17], at[B - 1]], [new] * 3, page)
        attend_close(a[rows], ref, mag, torch.bfloat16)
    run = step
    for i in range(4):
        check(i)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    run = graph.replay
    for i in (2, 0, 3, 1):
        check(i)


def test_two_streams_with_workspaces_of_their_own(P):
    pools, dev, c = make_cache(P, torch.bfloat16, [2000, 1500], 64, 4, seed=31, shared=10)
    q = torch.randn(2, 10, 16, D, generator=torch.Generator().manual_seed(9)).bfloat16()
    off = offsets_of([5, 5])
    ref = [ref_attend(x, pools, c.page_table.cpu(), [2000, 1500], [5, 5], 64) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    qd = q.to(DEV)
    ws = [c.attend_workspace(10, 16, 5, 10) for _ in range(2)]
    out = [torch.zeros(10, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            c.attend(qd[i], off, 5, shared_pages=10, workspace=ws[i], out=out[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        attend_close(out[i], *ref[i], torch.bfloat16)


def _stream_of(t):
    """The stream whose memory a tensor is, by the allocator's record."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_results_and_workspaces_are_memory_of_the_calls_stream(P):
    """With `stream`, what a call allocates is that stream's memory: filled again at once on the current stream, memory of
    the current one would change under the running call."""
    lengths = [9000 + 100 * i for i in range(8)]
    pools, dev, c = make_cache(P, torch.bfloat16, lengths, 64, 4, seed=35, shared=10)
    g = torch.Generator().manual_seed(12)
    q, k, v = (torch.randn(16, h, D, generator=g).bfloat16().to(DEV) for h in (16, 4, 4))
    off, cs = offsets_of([2] * 8), _table(10000, 128).to(DEV)
    pos = torch.zeros(1, 16, dtype=torch.int64, device=DEV)
    ref_q = c.append(k, v, off, q=q, cos_sin=cs)
    ref = c.attend(ref_q, off, 2, shared_pages=10)
    t, x = torch.rand(3, 4, 500, device=DEV), torch.zeros(3, 3, dtype=torch.int64, device=DEV)
    u, w, n = torch.rand(3, 3, device=DEV), torch.rand(3, device=DEV), torch.full((3,), 9, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    size = c.attend_workspace(16, 16, 2, 10).numel()
    for _ in range(10):
        a = c.append(k, v, off, q=q, cos_sin=cs, stream=s)
        b = c.attend(a, off, 2, shared_pages=10, stream=s)
        junk = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        del junk
        results = [a, b, *P.qk_norm_rope(q[None], k[None], pos, cs, stream=s), *P.draft_verify(t, None, x, u, w, lengths=n, stream=s),
                   c.attend_workspace(16, 16, 2, 10, stream=s)]
        torch.cuda.synchronize()
        assert [_stream_of(r) for r in results] == [s.cuda_stream] * len(results)
        assert torch.equal(a, ref_q) and torch.equal(b, ref)
    assert c.sync() == 0


def test_python_refusals(P):
    pools, dev, c = make_cache(P, torch.float16, [40, 33], 16, 2, seed=11, width=3)
    q, k = torch.zeros(3, 4, D, dtype=torch.float16, device=DEV), torch.zeros(3, 2, D, dtype=torch.float16, device=DEV)
    off = offsets_of([1, 2])
    cs = _table(64, 128).to(DEV)
    w = torch.ones(D, dtype=torch.float16, device=DEV)
    refusals = [
        lambda: c.attend(q.bfloat16(), off, 2), lambda: c.attend(q.cpu(), off, 2), lambda: c.attend(q[:, :3], off, 2),
        lambda: c.attend(q, off.long(), 2), lambda: c.attend(q, off[:2], 2), lambda: c.attend(q, off, 0),
        lambda: c.attend(q, off, 2, shared_pages=4), lambda: c.attend(q, off, 2, shared_pages=-1),
        lambda: c.attend(q, off, 2, softmax_scale=-1.0), lambda: c.attend(q, off, 2, softmax_scale=float("nan")),
        lambda: c.attend(q, off, 2, out=q[:2]), lambda: c.attend(q, off, 2, out=q),
        lambda: c.append(k, k, off, q=q, q_out=q), lambda: P.qk_norm_rope(q[None], k[None], None, q_out=q.view(1, 4, 3, D)), lambda: c.attend(q, off, 2, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
        lambda: c.attend(torch.zeros(3, 4, 2 * D, dtype=torch.float16, device=DEV)[..., ::2], off, 2),
        lambda: c.attend(torch.zeros(3 * 4 * D + 4, dtype=torch.float16, device=DEV)[4:].view(3, 4, D), off, 2),
        lambda: c.append(k, k[:2], off), lambda: c.append(k[:, :1], k[:, :1], off), lambda: c.append(k, k, off, q=q[:2]),
        lambda: c.append(k, k, off, q_out=q), lambda: c.append(k, k, off, cos_sin=cs[:, :24]),
        lambda: c.append(k, k, off, cos_sin=cs.half()), lambda: c.append(k, k, off, k_weight=w.float()),
        lambda: c.append(k, k, off, k_weight=w[:64]), lambda: c.append(k, k, off, eps=-1.0),
        lambda: c.append(k, k, off, cos_sin=cs, positions=torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: P.qk_norm_rope(q[None], k[None], None, cs), lambda: P.qk_norm_rope(q[None].float(), k[None].float(), None),
        lambda: P.qk_norm_rope(q[None], k[None, :2], None),
        lambda: P.PagedCache(dev[0], dev[1][:, :, :8], c.page_table, c.lengths),
        lambda: P.PagedCache(dev[0][:, :, :8], dev[1][:, :, :8], c.page_table, c.lengths),
        lambda: P.PagedCache(dev[0].float(), dev[1].float(), c.page_table, c.lengths),
        lambda: P.PagedCache(dev[0], dev[1], c.page_table.long(), c.lengths),
        lambda: P.PagedCache(dev[0], dev[1], c.page_table, c.lengths.int()),
        lambda: P.PagedCache(dev[0], dev[1], c.page_table, c.lengths[:1]),
        lambda: P.PagedCache(dev[0][:1].expand(4, -1, -1, -1), dev[1][:4], c.page_table, c.lengths),
    ]
    for i, f in enumerate(refusals):
        with pytest.raises((ValueError, P.PaluError)):
            f()
            pytest.fail(f"refusal {i} was accepted")
    torch.cuda.synchronize()
    assert c.sync() == 0
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, pools))
