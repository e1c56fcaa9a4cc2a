"""Attention over the 4-bit paged cache where the sizes of weights and value
scales lie far apart: one strong key over thousands of weak ones, scales down
to the smallest that fp16 has, large and small ones in one block.

Bar, as in tests/test_gpu_paged4.py: with the weights w and C = sum w (s c + |z|)
per output, (2^-10 + 2^-12) C + (eps / 2) |ref|, second-order terms by 1 + 2^-5.
To it comes what fp16 loses below its normal numbers, where a number is off by
half a step, 2^-25, or by itself, if that is less.  A weight is held relative to
a largest of 2^6 at least: sum min(w, 2^-31) (s c + |z|).  Its product with the
scale is held in units u in which the largest scale m of the block's 16 tokens
and the group lies in 2^-3 .. 2, but not below 2^-15: u <= max(8 m, 2^-15), so
sum min(w s, 2^-31 u) c; and a scale far under the block's largest is itself off:
sum w min(s, 2^-25 u) c.  (With more than 16 rows values enter as z + s c and only
the first of these applies.)
"""
import math

import pytest
import torch

from oracle import paged4_oracle as O4
from tests.test_gpu_paged4_step import DEV, DT, D, P, decode, offsets_of  # noqa: F401  (P: fixture)

pytestmark = pytest.mark.gpu


def values_of(codes, s):
    """Rows that are held as these codes (0 and 15 among each group's) and scales [tokens, heads, 4], exactly."""
    return (codes - 7.5) * s.double().repeat_interleave(32, -1)


def codes_like(tokens, heads, g):
    c = torch.randint(0, 16, (tokens, heads, D), generator=g, device=DEV).double()
    c[..., 0::32], c[..., 1::32] = 0, 15
    return c


def parts_of(cache, length):
    """Of sequence 0: keys, values, scales, zeros and codes of the values [length, Hk, 128] in 64 bits."""
    ids = cache.page_table[0, :-(-length // cache.page_size)].long()
    blocks = cache.pages[ids].unflatten(-1, (-1, O4.BLOCK)).transpose(1, 2).flatten(0, 1)
    flat = lambda x: x.transpose(1, 2).flatten(0, 1)[:length]
    k, v = (flat(decode(blocks, x)) for x in (False, True))
    scale = torch.from_numpy(O4.PLACES[3]).to(DEV)
    s, z = (flat(torch.stack([blocks[..., scale[..., i]], blocks[..., scale[..., i] + 1]], -1).view(torch.float16)[..., 0].double())
            .repeat_interleave(32, -1) for i in (0, 1))
    return k, v, s, z, torch.where(s > 0, (v - z) / torch.where(s > 0, s, 1.0), 0.0)


def check(cache, q, out, length):
    """q, out [Hq, 128] of sequence 0's last token."""
    k, v, s, z, c = (x.repeat_interleave(q.shape[0] // cache.kv_heads, 1) for x in parts_of(cache, length))
    w = torch.softmax(torch.einsum("hd,thd->ht", q.double(), k) * D ** -0.5, -1).T[..., None]
    ref, size = (w * v).sum(0), s * c + z.abs()
    m = torch.nn.functional.pad(s, (0, 0, 0, 0, 0, -length % 16)).view(-1, 16, *s.shape[1:]).amax(1).repeat_interleave(16, 0)[:length]
    u = torch.clamp(8 * m, min=2.0 ** -15)
    bar = (2.0 ** -10 + 2.0 ** -12) * (w * size).sum(0) + (w.clamp(max=2.0 ** -31) * size).sum(0) + \
        (torch.minimum(w * s, 2.0 ** -31 * u) * c).sum(0) + (w * torch.minimum(s, 2.0 ** -25 * u) * c).sum(0)
    eps = torch.finfo(out.dtype).eps
    bar = (1 + 2.0 ** -5) * bar + eps / 2 * ref.abs() + torch.finfo(out.dtype).smallest_normal * eps / 2
    worst = float(((out.double() - ref).abs() / bar).max())
    assert worst <= 1, worst


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq", [3, 12, 24])
@pytest.mark.parametrize("log_scale", [3, -9, -14, -18, -22])
def test_a_strong_key_over_thousands_of_weak_ones(P, dt, Hq, log_scale):
    """Each warp meets a strong key at once; its thousands of weak ones, 1.34 2^-12 each, weigh as much together.  What
    is lost of their products is lost alike in all of them."""
    dt, length, B, page = DT[dt], 65536, 152, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    table = torch.randperm(length // page, generator=g, device=DEV).int()[None].expand(B, -1).contiguous()
    pages = torch.zeros(length // page, 1, page * 160, dtype=torch.uint8, device=DEV)
    one = P.PagedCache4(pages, table[:1].contiguous(), torch.full((1,), length, device=DEV), page, dt)
    k = torch.zeros(length, 1, D, device=DEV)
    k[0:256:16] = (12 - math.log2(1.34)) * math.log(2) * D ** -0.5
    v = values_of(codes_like(length, 1, g), torch.full((length, 1, 4), 2.0 ** log_scale, device=DEV)).to(dt)
    one.append(k.to(dt), v, offsets_of([length]))
    assert torch.equal(one.read(offsets_of([length]), length)[1], v)
    cache = P.PagedCache4(pages, table, torch.full((B,), length, device=DEV), page, dt)
    q = (1 + torch.arange(Hq, device=DEV)[:, None] * 2.0 ** -6).expand(B, Hq, D).to(dt)
    out = cache.attend(q, offsets_of([1] * B), 1)
    for b in (0, 77, 151):
        check(cache, q[b], out[b], length)
    assert cache.sync() == 0


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hk", [(7, 1), (28, 2)])
@pytest.mark.parametrize("kind", ["blocks", "tokens", "groups", "rising", "falling", "outlier"])
def test_scales_far_apart(P, dt, Hq, Hk, kind):
    """Value scales from 2^-14 to 2^9, and the tokens with the small ones have all the weight: large and small ones in turn
    by blocks, within a block, by groups of channels, along the sequence; one token of 2^12 among them."""
    dt, length, page = DT[dt], 3000, 32
    g = torch.Generator(device=DEV).manual_seed(7)
    t = torch.arange(length, device=DEV)[:, None, None].expand(-1, Hk, 4)
    group = torch.arange(4, device=DEV).expand(length, Hk, -1)
    large = {"blocks": t // 16 % 2 == 1, "tokens": t % 3 == 1, "groups": group % 2 == 1, "rising": t > 1500, "falling": t < 1500,
             "outlier": t == 1000}[kind]
    log_scale = torch.where(large, {"outlier": 12.0, "tokens": -2.0}.get(kind, 9.0), -14.0)
    if kind in ("rising", "falling"):
        log_scale = torch.round(-14 + 23 * (t if kind == "rising" else length - 1 - t) / (length - 1))
    v = values_of(codes_like(length, Hk, g), 2.0 ** log_scale)
    weak = large.any(-1) if kind != "groups" else torch.zeros_like(large[..., 0])
    q = torch.randn(1, Hq, D, generator=g, device=DEV)
    lift = torch.where(weak, -1.0, 1.0)[..., None] * q[0].view(Hk, Hq // Hk, D).mean(1) * 4
    k = torch.randn(length, Hk, D, generator=g, device=DEV) / 2 + lift * (Hq // Hk) ** 0.5
    pages = torch.zeros(-(-length // page), Hk, page * 160, dtype=torch.uint8, device=DEV)
    table = torch.randperm(pages.shape[0], generator=g, device=DEV).int()[None].contiguous()
    cache = P.PagedCache4(pages, table, torch.full((1,), length, device=DEV), page, dt)
    cache.append(k.to(dt), v.to(dt), offsets_of([length]))
    q = q.to(dt)
    out = cache.attend(q, offsets_of([1]), 1)
    check(cache, q[0], out[0], length)
    assert torch.equal(out, cache.attend(q, offsets_of([1]), 1)) and cache.sync() == 0


@pytest.mark.parametrize("Hq", [3, 12, 24])
@pytest.mark.parametrize("fill", [-1, 0x7C00, 0xFC00 - 65536, 0x7E00])
def test_what_is_not_finite_stays_in_its_sequence(P, Hq, fill):
    """Every second sequence's scales and zeros are NaN or infinite (as no append writes them); a CTA takes both kinds one
    after the other."""
    B, length, page = 608, 300, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    width = -(-length // page)
    pages = torch.full((B * width, 1, page * 80), fill, dtype=torch.int16, device=DEV).view(torch.uint8)
    table = torch.randperm(B * width, generator=g, device=DEV).int().view(B, width)
    cache = P.PagedCache4(pages, table, torch.full((B,), length, device=DEV), page, torch.float16)
    good = P.PagedCache4(pages, table[1::2].contiguous(), torch.full((B // 2,), length, device=DEV), page, torch.float16)
    kv = torch.randn(B // 2 * length, 2, 1, D, generator=g, device=DEV).half()
    good.append(kv[:, 0], kv[:, 1], offsets_of([length] * (B // 2)))
    q = torch.randn(B, Hq, D, generator=g, device=DEV).half()
    out = cache.attend(q, offsets_of([1] * B), 1)
    assert bool(torch.isfinite(out[1::2]).all()) and (fill != -1 or bool(torch.isnan(out[::2]).all()))
    for b in (1, 3, 301, 607):
        one = P.PagedCache4(pages, table[b:b + 1].contiguous(), cache.lengths[:1], page, torch.float16)
        check(one, q[b], out[b], length)
    assert cache.sync() == 0


@pytest.mark.parametrize("Hq", [3, 12, 24])
def test_a_result_does_not_depend_on_what_others_hold(P, Hq):
    """Bit for bit, whatever scales the sequences have that a CTA takes before: each warp meets a strong key and then
    weak ones of 1.34 2^-19, whose products would round otherwise in other units, a few of the outputs with them."""
    B, length, page = 304, 4096, 128
    g = torch.Generator(device=DEV).manual_seed(11)
    width = -(-length // page)
    table = torch.randperm(B * width, generator=g, device=DEV).int().view(B, width)
    k = torch.zeros(B, length, 1, D, device=DEV)
    k[:, 0:256:16] = (19 - math.log2(1.34)) * math.log(2) * D ** -0.5
    v = values_of(codes_like(B * length, 1, g), torch.full((B * length, 1, 4), 2.0 ** -3, device=DEV)).half().view(B, length, 1, D)
    q = (1 + torch.arange(Hq, device=DEV)[:, None] * 2.0 ** -9).expand(B, Hq, D).half()
    outs = []
    for size in (1.0, 2.0 ** -3, 2.0 ** 9):
        mixed = v.clone()
        mixed[::2] *= size
        pages = torch.zeros(B * width, 1, page * 160, dtype=torch.uint8, device=DEV)
        cache = P.PagedCache4(pages, table, torch.full((B,), length, device=DEV), page, torch.float16)
        cache.append(k.half().view(-1, 1, D), mixed.view(-1, 1, D), offsets_of([length] * B))
        outs.append(cache.attend(q, offsets_of([1] * B), 1)[1::2])
        assert cache.sync() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
