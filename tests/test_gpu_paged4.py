"""The 4-bit paged cache (include/paged4.h) on the GPU: what an append writes,
byte by byte against the format's oracle; what a read gives back; attention of
new tokens over the pages against 64 bits, with and without a shared prefix.

Bars of the attention.  Scores carry fp32-accumulated products of inputs of size
a few, about 2^-16 absolute in the exponent, which enters every weight
relatively.  With few rows a KV head a weight p and its product p s with the
scale are each rounded to fp16 (2^-11); with w the weights and C = sum w (s c + |z|)
per output: |got - ref| <= (2^-10 + 2^-12) C + (eps / 2) |ref|.  With many rows
keys, values and weights are each rounded once to fp16 (2^-11): a key's rounding
moves its score by at most d_t = 2^-11 scale sum |q| |k|, so with A = sum w |v|
the bar gains sum w d |v| + |ref| sum w d, and weights and values cost 2^-11 A
each: |got - ref| <= (2^-10 + 2^-12) A + that + (eps / 2) |ref|.
Second-order terms are covered by 1 + 2^-5.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged4_oracle as O4

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


def table_of(n_pos, rope):
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rope // 2, dtype=torch.float64) / (rope // 2))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


class Case:
    """Sequences of these lengths in a pool whose unused bytes are `fill`; `layout`: the pool's strides."""

    def __init__(self, P, dt, lengths, page, Hk, seed=0, shared=0, width=None, fill=0xFF, layout="heads", spare=2, spread=1.0,
                 data=True):
        rng = np.random.default_rng(seed)
        B = len(lengths)
        width = width or max(1, -(-max(max(lengths), 1) // page))
        n_pages = B * width + spare
        ids = rng.permutation(n_pages)[:B * width].reshape(B, width).astype(np.int32)
        ids[:, :shared] = ids[0, :shared]
        self.dt, self.page, self.Hk, self.B, self.width = dt, page, Hk, B, width
        self.host = np.full((n_pages, Hk, page // 16, O4.BLOCK), fill, np.uint8)
        self.ids, self.lengths = ids, list(lengths)
        if data:
            self.fill_codes(rng, spread)
        self.pages = self.to_device(layout)
        self.table = torch.from_numpy(ids).to(DEV)
        self.len = torch.tensor(lengths, dtype=torch.int64, device=DEV)
        self.cache = P.PagedCache4(self.pages, self.table, self.len, page, dt)

    def fill_codes(self, rng, spread):
        """Random codes, scales and zeros for the tokens that the sequences have, whatever rows they might come from."""
        used = np.zeros(self.host.shape[:1] + (self.page,), bool)
        for b, n in enumerate(self.lengths):
            t = np.arange(n)
            used[self.ids[b, t // self.page], t % self.page] = True
        for p in np.nonzero(used.any(1))[0]:
            for t in np.nonzero(used[p])[0]:
                blk = self.host[p, :, t // 16]
                for values in (False, True):
                    place, scale = (O4.PLACES[2], O4.PLACES[3]) if values else (O4.PLACES[0], O4.PLACES[1])
                    code = rng.integers(0, 16, (self.Hk, D), dtype=np.uint8)
                    for high in (0, 4):
                        d = np.nonzero(place[t % 16, :, 1] == high)[0]
                        at = place[t % 16, d, 0]
                        blk[:, at] = blk[:, at] & (0xF0 if high == 0 else 0x0F) | code[:, d] << high
                    s = (rng.uniform(0.05, 0.3, (self.Hk, 4)) * spread).astype(np.float16)
                    z = (-7.5 * s.astype(np.float64) + rng.normal(0, 0.3, (self.Hk, 4)) * spread).astype(np.float16)
                    for x, j in ((s, 0), (z, 1)):
                        at = scale[t % 16, :, j]
                        raw = x.view(np.uint8).reshape(self.Hk, 4, 2)
                        blk[:, at], blk[:, at + 1] = raw[..., 0], raw[..., 1]

    def to_device(self, layout):
        x = torch.from_numpy(self.host.reshape(*self.host.shape[:2], -1))
        n, H, bytes_ = x.shape
        if layout == "heads":
            return x.to(DEV)
        if layout == "tokens":                                   # heads outermost
            return x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
        pool = torch.full((n, 2, H, bytes_ + 48), 0xEE, dtype=torch.uint8, device=DEV)   # a gap behind every page
        pool[:, 1, :, :bytes_] = x.to(DEV)
        return pool[:, 1, :, :bytes_]

    def rows(self, b, n=None):
        """Keys and values of a sequence, [n, Hk, 128] in 64 bits, from the host's copy."""
        n = self.lengths[b] if n is None else n
        blocks = self.host[self.ids[b]].transpose(0, 2, 1, 3).reshape(-1, self.Hk, O4.BLOCK)[:-(-n // 16)]
        return [O4.rows(blocks, v).transpose(0, 2, 1, 3).reshape(-1, self.Hk, D)[:n] for v in (False, True)]

    def size_rows(self, b, n):
        """s c + |z| of the values."""
        blocks = self.host[self.ids[b]].transpose(0, 2, 1, 3).reshape(-1, self.Hk, O4.BLOCK)[:-(-n // 16)]
        c, s, z = O4.parts(blocks, True)
        x = c.reshape(*c.shape[:-1], 4, 32) * s[..., None] + np.abs(z)[..., None]
        return x.reshape(c.shape).transpose(0, 2, 1, 3).reshape(-1, self.Hk, D)[:n]


def offsets_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)


def check_attend(case, q, new, got, scale=None, rows_behind=0, only=None):
    """got [N, Hq, 128] against the formula in 64 bits, with the bars above."""
    dt, Hk = case.dt, case.Hk
    q, got = q.cpu().double(), got.cpu().double()
    Hq, eps = q.shape[1], torch.finfo(dt).eps
    gq, scale = Hq // Hk, D ** -0.5 if scale is None else scale
    many = max(new) * gq > 16
    at, worst = 0, 0.0
    for b, n in enumerate(new):
        length = case.lengths[b]
        if n and (only is None or b in only):
            k, v = (torch.from_numpy(x).repeat_interleave(gq, 1) for x in case.rows(b))
            size = torch.from_numpy(case.size_rows(b, length)).repeat_interleave(gq, 1)
            x = q[at:at + n]
            s = torch.einsum("nhd,thd->hnt", x, k) * scale
            seen = torch.arange(length)[None] <= (length - n + torch.arange(n))[:, None]
            s.masked_fill_(~seen, -math.inf)
            w = torch.softmax(s, -1).nan_to_num(0.0)             # a row that sees nothing
            ref = torch.einsum("hnt,thd->nhd", w, v)
            bar = (2.0 ** -10 + 2.0 ** -12) * torch.einsum("hnt,thd->nhd", w, size)
            d = 2.0 ** -11 * scale * torch.einsum("nhd,thd->hnt", x.abs(), k.abs()) * seen
            A = torch.einsum("hnt,thd->nhd", w, v.abs())
            full = (2.0 ** -10 + 2.0 ** -12) * A + torch.einsum("hnt,thd->nhd", w * d, v.abs()) + \
                ref.abs() * (w * d).sum(-1).T[..., None]
            # which kernel takes a row follows from the whole call's sizes: either bar's kernel may have had it
            bar = torch.maximum(bar, full) if many or len(new) > 1 else bar
            bar = (1 + 2.0 ** -5) * bar + eps / 2 * ref.abs() + torch.finfo(dt).smallest_normal * eps
            err = (got[at:at + n] - ref).abs()
            worst = max(worst, float((err / bar).max()))
        at += n
    assert worst <= 1, worst
    return worst


# ------------------------------------------------------------------ append, read

@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("layout,page,new,lengths,Hq,Hk,rope,inter,norm", [
    ("heads", 16, (1,), (1,), 3, 1, 0, False, False), ("heads", 64, (1, 1, 1), (1, 16, 17), 8, 2, 128, False, True),
    ("tokens", 32, (5, 0, 31, 17), (9, 40, 33, 17), 10, 5, 64, True, True),
    ("gaps", 128, (130, 3), (260, 3), 7, 7, 48, False, False), ("heads", 16, (33, 16, 15), (40, 16, 31), 24, 8, 128, True, False),
    ("gaps", 16, (2, 64), (18, 80), 4, 4, 96, False, True), ("heads", 32, (47,), (1000,), 6, 6, 16, False, False)])
def test_append_and_read(P, dt, layout, page, new, lengths, Hq, Hk, rope, inter, norm):
    dt = DT[dt]
    g = torch.Generator().manual_seed(sum(lengths) + page)
    case = Case(P, dt, lengths, page, Hk, seed=page, fill=0xA5, layout=layout, data=False)
    N, pad = sum(new), 3                                          # rows behind the last sequence
    qkv = torch.randn(N + pad, Hq + 2 * Hk, D, generator=g).to(dt).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    cs = table_of(max(lengths) + 1, rope).to(DEV) if rope else None
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV) if norm else None for _ in range(2)]
    off = offsets_of(new)
    args = dict(cos_sin=cs, q_weight=w[0], k_weight=w[1], interleaved=inter)
    q4 = torch.full((N + pad, Hq, D), 7.0, dtype=dt, device=DEV)
    case.cache.append(k, v, off, q=q, q_out=q4, **args)
    assert case.cache.sync() == 0
    # an uncompressed cache says what rows are held
    pool = torch.zeros(2, case.host.shape[0], Hk, page, D, dtype=dt, device=DEV)
    plain = P.PagedCache(pool[0], pool[1], case.table, case.len)
    qp = torch.full_like(q4, 7.0)
    plain.append(k, v, off, q=q, q_out=qp, **args)
    assert torch.equal(q4, qp) and bool((q4[N:] == 7).all())
    rows = pool.float().cpu().numpy()
    want = case.host
    for b, (n, length) in enumerate(zip(new, lengths)):
        for t in range(length - n, length):
            p, i = case.ids[b, t // page], t % page
            for h in range(Hk):
                O4.write(want[p, h, i // 16], i % 16, rows[0, p, h, i], rows[1, p, h, i])
    assert np.array_equal(case.pages.cpu().numpy().reshape(want.shape), want)
    if layout == "gaps":
        base = case.pages._base if case.pages._base is not None else case.pages
        assert bool((base[:, 0] == 0xEE).all()) and bool((base[..., -48:] == 0xEE).all())
    # read back: the new tokens, rows behind them left alone
    ko, vo = (torch.full((N + pad, Hk, D), 9.0, dtype=dt, device=DEV) for _ in range(2))
    case.cache.read(off, N + pad, k_out=ko, v_out=vo)
    at = 0
    for b, n in enumerate(new):
        for got, ref in zip((ko, vo), case.rows(b)):
            ref = torch.from_numpy(ref[lengths[b] - n:]).float().to(dt)   # s c is exact in fp32, so z + s c is rounded to it once
            assert torch.equal(got[at:at + n].cpu(), ref)
        at += n
    assert bool((ko[N:] == 9).all()) and bool((vo[N:] == 9).all()) and case.cache.sync() == 0


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_values_of_every_kind(P, dt):
    """Rows without range, tiny and huge ranges, ties, zeros of either sign, infinities and NaN."""
    dt = DT[dt]
    g = torch.Generator().manual_seed(8)
    x = torch.randn(40, 3, D, generator=g)
    x[0] = 0
    x[1] = -0.0
    x[2] = 3.25
    x[3] *= 2.0 ** -20                                            # subnormal scales in fp16
    x[4] *= 2.0 ** -27
    x[5] *= 15000
    x[6, :, :] = torch.arange(D) % 32 / 2.0                       # ties: s = 15.5 / 15
    x[7, :, :] = (torch.arange(D) % 16).float()                   # s = 1
    x[7, :, 1::32] = 2.5
    x[8, 0, 5] = math.inf
    x[8, 1, 40] = -math.inf
    x[8, 2, 100] = math.nan
    x[9] = torch.linspace(-1, 1, D)
    x[12] = torch.linspace(-65504, 65504, D)
    x[13] = torch.linspace(60000, 65504, D)
    x[14] = torch.arange(D) % 31 * 0.5 - 7.5                      # z = -7.5 s: every second value on a border
    x[15] = x[14] * (1 + 2.0 ** -9)
    if dt == torch.bfloat16:
        x[10] *= 1e7                                              # scales and zeros that fp16 does not have
        x[11] *= 2e38
    x = x.to(dt)
    case = Case(P, dt, [40], 64, 3, data=False)
    off = offsets_of([40])
    case.cache.append(x.to(DEV), x.flip(1).contiguous().to(DEV), off)
    want = case.host
    for t in range(40):
        for h in range(3):
            O4.write(want[case.ids[0, 0], h, t // 16], t % 16, x[t, h].float().numpy(), x[t, 2 - h].float().numpy())
    got = case.pages.cpu().numpy().reshape(want.shape)
    assert np.array_equal(got, want)
    k, v = case.cache.read(off, 40)
    rk, rv = case.rows(0)
    for got, ref in ((k, rk), (v, rv)):
        ref = torch.from_numpy(ref).float().to(dt)
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref)) and torch.equal(got.cpu().nan_to_num(5.0), ref.nan_to_num(5.0))
    assert torch.isnan(k[8, 0, :32]).all() and torch.isfinite(k[8, 0, 32:]).all() and torch.isnan(k[8, 2, 96:]).all()


def test_an_append_token_by_token_is_one_of_a_chunk(P):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(75, 4, D, generator=g).half().to(DEV)
    a, b = (Case(P, torch.float16, [75], 32, 2, data=False, fill=0) for _ in range(2))
    a.cache.append(x[:, :2], x[:, 2:], offsets_of([75]))
    at = 0
    for n in (1, 15, 1, 7, 20, 1, 1, 29):
        b.len.fill_(at + n)
        b.cache.append(x[at:at + n, :2], x[at:at + n, 2:], offsets_of([n]))
        at += n
    assert torch.equal(a.pages, b.pages) and a.cache.sync() == 0 and b.cache.sync() == 0


def test_lengths_of_sequences_without_new_tokens_do_not_matter(P):
    g = torch.Generator().manual_seed(6)
    x = torch.randn(9, 2, D, generator=g).half().to(DEV)
    case, other = (Case(P, torch.float16, [20, 30, 20], 16, 1, data=False, fill=0) for _ in range(2))
    for bad in (-5, 1 << 40):
        case.len[1] = bad
        case.cache.append(x[:, :1], x[:, 1:], offsets_of([4, 0, 5]))
        k, v = case.cache.read(offsets_of([4, 0, 5]), 9)
        assert case.cache.sync() == 0
    other.cache.append(x[:, :1], x[:, 1:], offsets_of([4, 0, 5]))
    assert torch.equal(case.pages, other.pages)
    assert all(torch.equal(a, b) for a, b in zip((k, v), other.cache.read(offsets_of([4, 0, 5]), 9)))


def test_read_from_given_places(P):
    case = Case(P, torch.float16, [50, 7, 200], 32, 2)
    starts = torch.tensor([3, 0, 111], dtype=torch.int64, device=DEV)
    off = offsets_of([40, 0, 60])
    k, v = case.cache.read(off, 100, starts=starts)
    for at, b, first, n in ((0, 0, 3, 40), (40, 2, 111, 60)):
        for got, ref in zip((k, v), case.rows(b)):
            assert torch.equal(got[at:at + n].cpu(), torch.from_numpy(ref[first:first + n]).float().half())
    assert case.cache.sync() == 0


def test_append_and_read_refused_on_the_device(P):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(12, 4, D, generator=g).half().to(DEV)
    for kind, bit in (("span", 128), ("capacity", 1), ("page", 64), ("position", 256), ("order", 128), ("rows", 128)):
        case = Case(P, torch.float16, [20, 20, 20], 16, 1, data=False, fill=0x11)
        new, off, cs = [4, 4, 4], offsets_of([4, 4, 4]), None
        if kind == "span":
            case.len[1] = 3
        elif kind == "capacity":
            case.len[1] = 33
        elif kind == "page":
            case.table[1, 1] = case.host.shape[0]
        elif kind == "position":
            cs = table_of(19, 32).to(DEV)                        # the last token's place is 19
        elif kind == "order":
            off[2] = 3
        else:
            off[3] = 13
        q = case.cache.append(x[:, 1:2], x[:, 2:3], off, q=x[:, :1], cos_sin=cs)
        with pytest.raises(P.PaluError, match="device error word"):
            case.cache.sync()
        untouched = torch.full_like(case.pages, 0x11)
        if kind in ("span", "capacity", "page"):
            assert torch.isnan(q[4:8]).all() and torch.isfinite(q[:4]).all() and torch.isfinite(q[8:]).all()
            # the other sequences' pages, with the refused one as if it brought nothing
            other = Case(P, torch.float16, [20, 20, 20], 16, 1, data=False, fill=0x11)
            other.cache.append(torch.cat([x[:4], x[8:]])[:, 1:2], torch.cat([x[:4], x[8:]])[:, 2:3], offsets_of([4, 0, 4]))
            assert torch.equal(case.pages, other.pages) and not torch.equal(case.pages, untouched)
        if kind == "position":
            assert torch.isnan(q[3::4]).all() and torch.isfinite(q[:3]).all()
        k = torch.full((12, 1, D), 5.0, dtype=torch.float16, device=DEV)
        v = k.clone()
        case.cache.read(off, 12, k_out=k, v_out=v)
        if kind != "position":
            with pytest.raises(P.PaluError, match="device error word"):
                case.cache.sync()
        if kind in ("span", "capacity", "page"):
            assert bool((k[4:8] == 5).all()) and bool((v[4:8] == 5).all()) and not bool((k[:4] == 5).any())


# ------------------------------------------------------------------ attention

ATTEND = [
    (16, (1,), (1,), 1, 1, 0), (16, (1,), (513,), 24, 8, 0), (32, (1, 1, 1), (5, 16, 17), 8, 2, 0),
    (64, (1,) * 5, (130, 1, 128, 64, 2000), 28, 4, 0), (16, (2, 1, 2), (40, 300, 2), 12, 3, 0),
    (128, (5, 3, 1), (700, 3, 129), 28, 4, 0), (32, (3, 0, 1), (65, 90, 1), 5, 1, 0), (64, (1,) * 3, (100, 1000, 3000), 16, 16, 0),
    (16, (17, 40), (17, 90), 8, 8, 0), (64, (64, 1, 33), (64, 200, 900), 24, 8, 0), (128, (200,), (450,), 6, 2, 0),
    (32, (1,) * 6, (190, 200, 161, 400, 777, 163), 24, 8, 5), (16, (2,) * 4, (130, 140, 200, 129), 7, 1, 8),
    (64, (1, 5, 2, 5), (400, 500, 330, 700), 28, 4, 5), (64, (40, 1, 17), (640, 577, 700), 16, 4, 9),
    (16, (1,) * 40, tuple(513 + 7 * i for i in range(40)), 28, 4, 32)]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lengths,Hq,Hk,shared", ATTEND)
def test_attend(P, dt, page, new, lengths, Hq, Hk, shared):
    case = Case(P, DT[dt], lengths, page, Hk, seed=len(lengths) + page, shared=shared)
    g = torch.Generator().manual_seed(page)
    N = sum(new)
    q = torch.randn(N + 2, Hq + 3, D, generator=g).to(DT[dt]).to(DEV)[:, 1:Hq + 1]
    out = torch.full((N + 2, Hq, D), 7.0, dtype=DT[dt], device=DEV)
    case.cache.attend(q, offsets_of(new), max(new), shared_pages=shared, out=out)
    assert case.cache.sync() == 0 and bool((out[N:] == 7).all())
    check_attend(case, q[:N], new, out[:N])
    again = case.cache.attend(q, offsets_of(new), max(new), shared_pages=shared)
    assert torch.equal(again[:N], out[:N])


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("new", [(1, 4, 1), (40, 25, 1)])
@pytest.mark.parametrize("shared", [0, 1])
def test_rows_that_see_nothing_are_zero(P, dt, new, shared):
    lengths = [0, 3, 20]
    case = Case(P, DT[dt], [max(n, 1) for n in lengths], 16, 2, shared=shared)
    case.lengths = lengths
    case.len.copy_(torch.tensor(lengths))
    q = torch.randn(sum(new), 6, D, device=DEV).to(DT[dt])
    out = case.cache.attend(q, offsets_of(new), max(new), shared_pages=shared)
    a = new[0]
    assert case.cache.sync() == 0 and bool((out[:a] == 0).all())
    assert bool((out[a:a + new[1] - 3] == 0).all()) and bool((out[a + new[1] - 3:] != 0).any())
    check_attend(case, q, new, out, only=(1, 2))


@pytest.mark.parametrize("new", [1, 7, 40])
def test_sizes_of_scales_and_queries(P, new):
    """Value scales from the smallest to the largest that fp16 has, queries of any size, one large weight among many."""
    for spread, qsize in ((1.0, 1e-3), (2.0 ** -9, 1.0), (2.0 ** 12, 1e-3), (1.0, 30.0), (30.0, 0.1)):
        case = Case(P, torch.float16, [900, new + 1], 64, 2, spread=spread, seed=3)
        q = (torch.randn(2 * new, 6, D, device=DEV) * qsize).half()
        out = case.cache.attend(q, offsets_of([new, new]), new)
        check_attend(case, q, [new, new], out)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_scales_that_grow_along_the_sequence(P, dt):
    """Value scales far above 1 behind small ones: the weights' range has to follow."""
    case = Case(P, DT[dt], [600], 32, 1, seed=5)
    blocks = case.host[case.ids[0]].reshape(-1, O4.BLOCK)
    for t in range(600):
        for j in range(4):
            at, zat = O4.value_scale_place(t % 16, j)
            f = 2.0 ** (t // 64 + (3 if t % 50 == 7 else 0))
            blk = case.host[case.ids[0, t // 32], 0, t % 32 // 16]
            for a in (at, zat):
                x = np.frombuffer(blk[a:a + 2].tobytes(), np.float16)[0]
                blk[a:a + 2] = np.frombuffer(np.float16(np.float64(x) * f).tobytes(), np.uint8)
    del blocks
    case.pages.copy_(torch.from_numpy(case.host.reshape(*case.host.shape[:2], -1)))
    q = torch.randn(1, 7, D, device=DEV).to(DT[dt])
    check_attend(case, q, [1], case.cache.attend(q, offsets_of([1]), 1))


def test_scores_far_below_zero(P):
    """Queries of 2^120: every score of a row below -1e30, or every one above 1e30, and one key has all the weight."""
    case = Case(P, torch.bfloat16, [60], 16, 1, seed=2, data=False, fill=0)
    g = torch.Generator().manual_seed(8)
    x, y = torch.rand(60, 1, D, generator=g) + 1, torch.randn(60, 1, D, generator=g)
    case.cache.append(x.bfloat16().to(DEV), y.bfloat16().to(DEV), offsets_of([60]))
    case.host = case.pages.cpu().numpy().reshape(case.host.shape)
    k, v = (torch.from_numpy(a)[:, 0] for a in case.rows(0))
    q = torch.full((1, 2, D), 2.0 ** 120, dtype=torch.bfloat16)
    q[0, 1] *= -1
    out = case.cache.attend(q.to(DEV), offsets_of([1]), 1).cpu().double()
    sums = k.sum(1)
    for h, at, other in ((0, sums.argmax(), sums.topk(2).values), (1, sums.argmin(), sums.topk(2, largest=False).values)):
        assert (other[0] - other[1]).abs() > 2.0 ** -18 * sums.max()              # fp32's sums tell them apart
        bar = (2.0 ** -8 + 2.0 ** -9) * torch.from_numpy(case.size_rows(0, 60))[at, 0]   # bf16's rounding, and the weight's
        assert ((out[0, h] - v[at]).abs() <= bar).all()


def test_softmax_scale_and_zero_queries(P):
    case = Case(P, torch.bfloat16, [300, 70], 16, 2)
    q = torch.randn(2, 4, D, device=DEV).bfloat16()
    q[0, 1] = 0
    check_attend(case, q, [1, 1], case.cache.attend(q, offsets_of([1, 1]), 1, softmax_scale=0.3), scale=np.float32(0.3))


def test_what_lies_behind_the_lengths_does_not_matter(P):
    """Unused bytes of all ones are NaN scales and zeros."""
    for new in (1, 9, 50):
        outs = []
        for fill in (0xFF, 0x00, 0x7C):
            case = Case(P, torch.float16, [77, new, 131], 64, 2, seed=9, fill=fill, shared=0)
            g = torch.Generator().manual_seed(4)
            q = torch.randn(3 * new, 6, D, generator=g).half().to(DEV)
            outs.append(case.cache.attend(q, offsets_of([new] * 3), new))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and torch.isfinite(outs[0]).all()


def test_attend_refused_on_the_device(P):
    for kind, bit in (("span", 128), ("capacity", 1), ("page", 64), ("new", 128)):
        case = Case(P, torch.float16, [40, 40, 40], 16, 1)
        q = torch.randn(3, 4, D, device=DEV).half()
        off = offsets_of([1, 1, 1])
        if kind == "span":
            off[2] = 0
        elif kind == "capacity":
            case.len[1] = 49
        elif kind == "page":
            case.table[1, 2] = -1
        else:
            q = torch.randn(4, 4, D, device=DEV).half()
            off = offsets_of([1, 2, 1])
        out = case.cache.attend(q, off, 1)
        with pytest.raises(P.PaluError, match="device error word"):
            case.cache.sync()
        check_attend(case, q[:1], [1], out[:1], only=(0,))


def test_captured_steps_follow_lengths_and_pages(P):
    """A captured step of append and attention, replayed while lengths, offsets and pages change."""
    case = Case(P, torch.bfloat16, [1, 1], 16, 2, width=8, data=False, fill=0)
    N, Hq = 6, 4
    x = torch.zeros(N, Hq + 4, D, dtype=torch.bfloat16, device=DEV)
    off = offsets_of([1, 1])
    ws = case.cache.attend_workspace(N, Hq, 4)
    out, q4 = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device=DEV), torch.zeros(N, Hq, D, dtype=torch.bfloat16, device=DEV)
    kr, vr = (torch.zeros(N, 2, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        case.cache.append(x[:, Hq:Hq + 2], x[:, Hq + 2:], off, q=x[:, :Hq], q_out=q4)
        case.cache.attend(q4, off, 4, workspace=ws, out=out)
        case.cache.read(off, N, k_out=kr, v_out=vr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(0)
    case.len.zero_()
    lengths = [0, 0]
    for new in ((4, 2), (1, 4), (0, 3), (4, 1), (3, 3), (1, 0)):
        lengths = [a + b for a, b in zip(lengths, new)]
        case.len.copy_(torch.tensor(lengths))
        off.copy_(offsets_of(new))
        x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        n = sum(new)
        case.host = case.pages.cpu().numpy().reshape(case.host.shape)
        case.lengths = lengths
        check_attend(case, q4[:n], new, out[:n])
        at = 0
        for b, m in enumerate(new):
            for got, ref in zip((kr, vr), case.rows(b)):
                assert torch.equal(got[at:at + m].cpu(), torch.from_numpy(ref[lengths[b] - m:]).float().bfloat16())
            at += m
    assert case.cache.sync() == 0


def test_two_streams(P):
    cases = [Case(P, torch.float16, [3000, 100], 64, 2, seed=i) for i in range(2)]
    q = [torch.randn(2, 8, D, device=DEV).half() for _ in range(2)]
    off = offsets_of([1, 1])
    want = [c.cache.attend(x, off, 1) for c, x in zip(cases, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [c.cache.attend(x, off, 1, stream=s) for c, x, s in zip(cases, q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_beyond_32_bits_in_a_large_pool(P):
    """The last pages of a pool of 5 GB."""
    page, Hk = 128, 4
    n_pages = 5 * 10 ** 9 // (Hk * page * 160)
    pages = torch.empty(n_pages, Hk, page * 160, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([300], dtype=torch.int64, device=DEV)
    cache = P.PagedCache4(pages, table, lengths, page, torch.float16)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(300, 3 * Hk, D, generator=g).half().to(DEV)
    off = offsets_of([300])
    cache.append(x[:, Hk:2 * Hk], x[:, 2 * Hk:], off)
    k, v = cache.read(off, 300)
    for got, ref in ((k, x[:, Hk:2 * Hk]), (v, x[:, 2 * Hk:])):
        assert torch.equal(got.cpu(), torch.from_numpy(O4.held(ref.float().cpu().numpy())).float().half())
    one = offsets_of([1])
    out = cache.attend(x[:1, :Hk], one, 1)
    s = torch.einsum("hd,thd->ht", x[0, :Hk].double(), k.double()) * D ** -0.5
    ref = torch.einsum("ht,thd->hd", torch.softmax(s, -1), v.double())
    assert float((out[0].double() - ref).norm() / ref.norm()) < 2e-3 and cache.sync() == 0


def test_python_refusals(P):
    case = Case(P, torch.float16, [20, 3], 16, 2)
    q, k = torch.zeros(2, 4, D, dtype=torch.float16, device=DEV), torch.zeros(2, 2, D, dtype=torch.float16, device=DEV)
    off = offsets_of([1, 1])
    for bad in (lambda: P.PagedCache4(case.pages[..., :-16], case.table, case.len, 16, torch.float16),
                lambda: P.PagedCache4(case.pages.view(torch.int8), case.table, case.len, 16, torch.float16),
                lambda: P.PagedCache4(case.pages, case.table, case.len, 32, torch.float16),
                lambda: P.PagedCache4(case.pages, case.table, case.len, 16, torch.float32),
                lambda: P.PagedCache4(case.pages.cpu(), case.table, case.len, 16, torch.float16),
                lambda: P.PagedCache4(case.pages, case.table.long(), case.len, 16, torch.float16),
                lambda: P.PagedCache4(case.pages, case.table, case.len[:1], 16, torch.float16),
                lambda: case.cache.append(k.bfloat16(), k, off), lambda: case.cache.append(k, k, off.long()),
                lambda: case.cache.append(k[:, :1], k, off), lambda: case.cache.attend(q.float(), off, 1),
                lambda: case.cache.read(off, 2, starts=case.len.int()),
                lambda: case.cache.read(off, 2, k_out=torch.zeros(3, 2, D, dtype=torch.float16, device=DEV)),
                lambda: case.cache.attend(q, off, 1, workspace=torch.zeros(4, dtype=torch.float32, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: case.cache.attend(q, off, 0), lambda: case.cache.attend(q[:, :3], off, 1),
                lambda: case.cache.attend(q, off, 1, shared_pages=9),
                lambda: case.cache.attend(q, off, 1, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
                lambda: case.cache.attend(q, off, 1, out=q), lambda: case.cache.read(off, 2, k_out=k, v_out=k)):
        with pytest.raises(P.PaluError):
            bad()
