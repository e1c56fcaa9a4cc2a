"""Plans of many rows, which a cluster of CTAs takes (include/pages.h): captured
and replayed, refused in between, and two pools at once."""
import numpy as np
import pytest
import torch

from tests.test_gpu_pages import DEV, P, make, same  # noqa: F401  (P: fixture)

pytestmark = pytest.mark.gpu


def test_a_captured_plan_of_many_rows(P):
    B, tokens = 600, 9000
    pool, plain = make(P, B, 12, 16, 4000)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    bufs = dict(offsets=torch.zeros(B + 1, dtype=torch.int32, device=DEV), positions=torch.zeros(tokens, dtype=torch.int64, device=DEV),
                slots=torch.zeros(tokens, dtype=torch.int64, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.plan(new, tokens, **bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.plan(new, tokens, **bufs)
    rng = np.random.default_rng(0)
    refused = 0
    for step in range(12):
        n = rng.integers(0, 30 if step != 5 else 40, B)            # the 6th brings more rows than there are
        if step % 2:
            plain.lengths = [int(rng.integers(0, x + 1)) for x in plain.lengths]
            pool.lengths.copy_(torch.tensor(plain.lengths))
        new.copy_(torch.tensor(n))
        graph.replay()
        torch.cuda.synchronize()
        want = plain.plan([int(x) for x in n], tokens)
        same(pool, plain, (bufs["offsets"], bufs["positions"], bufs["slots"]), want)
        assert pool.error.item() == want[3]
        refused += want[3] != 0
        pool.error.zero_()
    assert 0 < refused < 12


def test_two_pools_on_two_streams(P):
    pairs = [make(P, 700, 10, 16, 5000) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    rng = np.random.default_rng(1)
    torch.cuda.synchronize()
    for step in range(6):
        news = [rng.integers(0, 25, 700) for _ in pairs]
        dev = [torch.tensor(n, dtype=torch.int32, device=DEV) for n in news]
        torch.cuda.synchronize()
        got = [pool.plan(d, 20000, stream=s) for (pool, _), d, s in zip(pairs, dev, streams)]
        torch.cuda.synchronize()
        for (pool, plain), n, g in zip(pairs, news, got):
            want = plain.plan([int(x) for x in n], 20000)
            same(pool, plain, g, want)
            assert pool.error.item() == want[3]
            pool.error.zero_()
