"""Attention behind a shared prefix, at sizes for which the shared pages are read
once.  That they were is part of each test: in a second call the other
sequences' leading table entries name a page of NaN, which only a call that
reads row 0's pages leaves out of its result.  Bars as in test_gpu_paged.py."""
import math

import pytest
import torch

from test_gpu_paged import D, DEV, DT, attend_close, make_cache, offsets_of, ref_attend

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
