"""Weights of the paged attention far below the largest one, of which there are
many: each counts for nothing, their sum does not."""
import math

import pytest
import torch

from test_gpu_paged import D, DEV, DT, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from rank_latent_kv_gb300 import palu
    palu.lib()
    return palu


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,heads,S,shared", [(304, 2, 1200000, 0), (304, 10, 1200000, 0), (2, 2, 400000, 2000)])
def test_weights_below_the_steps_of_fp16(P, dt, B, heads, S, shared):
    """A first token whose weight is 2^25.3 .. 2^26.5 times every other's: below half the smallest fp16 number where the
    largest weight is 1, and together 0.6 to 2 % of the result.  In up to 8 and up to 16 rows; sequences enough that one
    CTA, with a running maximum a warp, has all of a sequence; and with shared pages.  All sequences name the same pages."""
    d, page = DT[dt], 128
    g = torch.Generator().manual_seed(5)
    width = S // page
    k, v = torch.zeros(width, 1, page, D), 1 + torch.randn(width, 1, page, D, generator=g)
    # scores: 128 channels of 0.25 * key / sqrt(128); the first token's is far above the others'
    gap = 25.3 + 1.2 * torch.rand(width, page, generator=g)
    k[:, 0] = (40.0 - gap * math.log(2) * math.sqrt(D) / (D * 0.25))[..., None]
    k[0, 0, 0] = 40.0
    k, v = k.to(d), v.to(d)
    q = torch.full((B, heads, D), 0.25).to(d)
    kd, vd = k.to(DEV), v.to(DEV)
    table = torch.arange(width, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    c = P.PagedCache(kd, vd, table, torch.full((B,), S, device=DEV))
    out = c.attend(q.to(DEV), offsets_of([1] * B), 1, shared_pages=shared)
    assert c.sync() == 0
    kd, vd = kd.double().view(-1, D)[:S], vd.double().view(-1, D)[:S]
    p = torch.softmax(kd.sum(1) * 0.25 / math.sqrt(D), 0)
    assert 0.002 < float(p[1:].sum()) < 0.03
    ref, mag = (p @ vd).cpu(), (p @ vd.abs()).cpu()
    eps = torch.finfo(d).eps
    # scores of 113 with 128 products of size 10 / sqrt(128): fp32 sums are right to about 128 * 113 * 2^-24 = 2^-10 at
    # worst, which enters through the other tokens' 3 % at most; the rest as in test_gpu_paged.py
    # And the accumulators: of a sequence that one CTA has, each of its eight warps takes 16 keys of every 128 and adds two
    # products of them (weights rounded, and their remainders) to an fp32 number, each addition right to one step, 2^-23 of
    # it, however it rounds; the accumulator is at most A.  So S / 128 * 2 * 2^-23 * A (0.2 % at 1,200,000 tokens).
    bar = (eps / 2 + 2.0 ** -12 + S / 128 * 2.0 ** -22) * mag + eps / 2 * ref.abs()
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= bar).all()), float((err / bar).max())
