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


@pytest.mark.parametrize("Hq,Hk,new", [(24, 8, 1), (16, 2, 2)])
def test_a_captured_call_follows_the_lengths(P, Hq, Hk, new):
    """One graph, replayed as own tokens come and go: the division of the CTAs between prefix and own keys is the device's."""
    B, page, shared, own = 96, 64, 48, 700
    prefix = shared * page
    cache = filled(P, torch.float16, B, Hk, page, prefix + own, shared=shared, seed=4)
    g = torch.Generator(device=DEV).manual_seed(6)
    q = torch.randn(B * new, Hq, D, generator=g, device=DEV).half()
    off, ws, out = offsets_of([new] * B), cache.attend_workspace(B * new, Hq, new, shared), torch.zeros_like(q)

    def call():
        cache.attend(q, off, new, shared_pages=shared, workspace=ws, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([prefix + own] * B, [prefix] * B, [prefix // 2 + i for i in range(B)], [prefix + own if i == 7 else 1 + i for i in range(B)],
                    [0] * (B - 1) + [prefix + 5], [prefix + 1 + 7 * i for i in range(B)]):
        lengths = [n if n == 0 else max(n, new) for n in lengths]
        cache.lengths.copy_(torch.tensor(lengths))
        graph.replay()
        torch.cuda.synchronize()
        check(cache, q, [new] * B, out, lengths, only=(0, 7, 40, B - 1))
        for b in range(B):
            if lengths[b] == 0:
                assert bool((out[b * new:(b + 1) * new] == 0).all())
    assert cache.sync() == 0


def test_two_streams_behind_one_prefix(P):
    B, Hq, Hk, page, shared, own = 64, 24, 8, 32, 128, 300
    cache = filled(P, torch.bfloat16, B, Hk, page, shared * page + own, shared=shared, seed=8)
    qs = [torch.randn(B, Hq, D, device=DEV).bfloat16() for _ in range(2)]
    off = offsets_of([1] * B)
    want = [cache.attend(q, off, 1, shared_pages=shared) for q in qs]
    ws = [cache.attend_workspace(B, Hq, 1, shared) for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, w, o, s in zip(qs, ws, outs, streams):
            cache.attend(q, off, 1, shared_pages=shared, workspace=w, out=o, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert cache.sync() == 0
