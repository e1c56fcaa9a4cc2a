"""Decode of many sequences behind a long shared prefix over the 4-bit paged
cache: more sequences than a warp has lanes, than a CTA has threads, and with
own tokens of every number, so that each thread of the plan holds a part of
the line.

Bars: those of tests/test_gpu_paged4_step.py, a norm over each output row.
"""
import pytest
import torch

from tests.test_gpu_paged4_step import BAR, DEV, DT, D, P, check, filled, offsets_of  # noqa: F401  (P: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,Hq,Hk,page,shared,own,new", [
    (64, 24, 8, 64, 64, 400, 1), (700, 8, 4, 64, 32, 130, 1), (300, 12, 2, 64, 32, 257, 2), (1500, 8, 1, 16, 128, 40, 1)])
def test_hundreds_of_sequences_behind_a_prefix(P, dt, B, Hq, Hk, page, shared, own, new):
    prefix = shared * page
    cache = filled(P, DT[dt], B, Hk, page, prefix + own, shared=shared, seed=B)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(B * new, Hq, D, generator=g, device=DEV).to(DT[dt])
    off = offsets_of([new] * B)
    some = (0, 31, 32, 33, B // 3, B // 2, B - 2, B - 1)
    # all long; every length from the prefix to its own end, in no order; many that bring nothing of their own
    for lengths in ([prefix + own] * B, [prefix + new + i * 37 % (own - new + 1) for i in range(B)],
                    [prefix + (own if i % 50 == 49 else 0) for i in range(B)]):
        cache.lengths.copy_(torch.tensor(lengths))
        out = cache.attend(q, off, new, shared_pages=shared)
        check(cache, q, [new] * B, out, lengths, only=some)
        alone = cache.attend(q, off, new)
        err = (out.float() - alone.float()).norm(dim=-1) / alone.float().norm(dim=-1)
        assert float(err.max()) < 2 * BAR[DT[dt]], float(err.max())
        for _ in range(10):
            assert torch.equal(out, cache.attend(q, off, new, shared_pages=shared))
    assert cache.sync() == 0
