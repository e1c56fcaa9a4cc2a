"""Host side of include/paged4.h, include/pages.h and include/rope.h without a
GPU: the structs match the headers, and every argument that a call can refuse
is refused with a status and a message before anything is launched."""
import ctypes
import math
import os
import subprocess
import tempfile

import pytest

from tests.conftest import ROOT
from tests.test_abi import palu  # noqa: F401  (fixture)

I64x2 = ctypes.c_int64 * 2
A = 1 << 20            # aligned addresses that are never read
FAR = 1 << 30


def test_struct_layouts_match_the_headers(palu):
    prog = r'''
#include <stdio.h>
#include <stddef.h>
#include "paged4.h"
#include "pages.h"
#include "rope.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %d\n", sizeof(palu_paged4_cache), offsetof(palu_paged4_cache, strides),
         offsetof(palu_paged4_cache, error), sizeof(palu_page_pool), offsetof(palu_page_pool, page_table),
         offsetof(palu_page_pool, error), sizeof(palu_rope_scaling), offsetof(palu_rope_scaling, base),
         offsetof(palu_rope_scaling, magnitude), PALU_PAGED4_BLOCK);
  printf("%d %d %d %d\n", PALU_ROPE_PLAIN, PALU_ROPE_LINEAR, PALU_ROPE_NTK, PALU_ROPE_PARTS);
  return 0;
}'''
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(src, "w") as f:
            f.write(prog)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        vals = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    c, p, r = palu.palu_paged4_cache, palu.palu_page_pool, palu.palu_rope_scaling
    assert vals[:10] == [ctypes.sizeof(c), c.strides.offset, c.error.offset, ctypes.sizeof(p), p.page_table.offset, p.error.offset,
                         ctypes.sizeof(r), r.base.offset, r.magnitude.offset, palu.PALU_PAGED4_BLOCK]
    packed = palu._pack_rope(1, 2, 3.0, 4.0, 5.0, 6.0, 7.0, 8.0)
    x = r.from_buffer_copy(packed)
    assert len(packed) == ctypes.sizeof(r) and (x.kind, x.rope_dim, x.base, x.magnitude) == (1, 2, 3.0, 8.0)
    assert vals[10:] == [palu.PALU_ROPE_KINDS[k] for k in ("plain", "linear", "ntk", "parts")]


def init(palu, dtype=0, hk=2, page=32, n_pages=8, pages=A, strides=(10240, 5120), table=A, batch=3, width=4, lengths=A, error=A):
    c = palu.palu_paged4_cache()
    st = palu.lib().palu_paged4_cache_init(ctypes.byref(c), dtype, hk, page, n_pages, pages, I64x2(*strides), table, batch, width,
                                           lengths, error)
    return st, c


def test_cache_init(palu):
    st, c = init(palu)
    assert st == 0 and (c.kv_heads, c.page_size, c.batch, c.table_width, c.n_pages) == (2, 32, 3, 4, 8)
    for bad in (dict(dtype=2), dict(hk=0), dict(page=24), dict(page=256), dict(n_pages=0), dict(n_pages=1 << 31), dict(pages=0),
                dict(pages=A + 8), dict(strides=(10240, 5128)), dict(strides=(-10240, 5120)), dict(strides=(0, 5120)),
                dict(strides=(1 << 39, 5120)), dict(n_pages=(1 << 31) - 1, strides=(1 << 38, 5120)), dict(table=0), dict(table=A + 2), dict(batch=0), dict(batch=4097), dict(width=0),
                dict(width=(1 << 25) + 1), dict(lengths=0), dict(lengths=A + 4), dict(error=0), dict(error=A + 1)):
        st, c = init(palu, **bad)
        assert st in (1, 2) and c.magic == 0 and palu.palu_last_error(), bad


def test_workspace_size(palu):
    _, c = init(palu)
    n = ctypes.c_size_t()
    size = lambda *a: palu.lib().palu_paged4_attn_workspace_size(ctypes.byref(c), *a, ctypes.byref(n))
    assert size(3, 4, 1, 0) == 0 and n.value > 0 and n.value % 256 == 0
    for bad in ((0, 4, 1, 0), (3, 0, 1, 0), (3, 3, 1, 0), (3, 4, 0, 0), (3, 4, 1, 5), (3, 4, 1, -1), (3, 130, 1, 0), (1 << 30, 4, 1, 0)):
        assert size(*bad) in (1, 2), bad
    assert palu.lib().palu_paged4_attn_workspace_size(ctypes.byref(palu.palu_paged4_cache()), 3, 4, 1, 0, ctypes.byref(n)) == 4


@pytest.mark.parametrize("width", [4, 40])
def test_a_workspace_serves_smaller_calls(palu, width):
    _, c = init(palu, width=width, batch=30)
    n = ctypes.c_size_t()

    def size(tokens, new, shared):
        assert palu.lib().palu_paged4_attn_workspace_size(ctypes.byref(c), tokens, 14, new, shared, ctypes.byref(n)) == 0
        return n.value
    sizes = [(t, m) for t in (1, 2, 3, 30, 100, 300) for m in (1, 2, 3, 10, 100)]
    for t, m in sizes:
        shared = {size(t, m, s) for s in range(1, width + 1)}
        assert len(shared) == 1 and size(t, m, 0) <= shared.pop()
        for t1, m1 in sizes:
            if t1 <= t and m1 <= m:
                assert all(size(t1, m1, s) <= size(t, m, s) for s in (0, 1, width // 2, width))


def attend(palu, c, tokens=3, offsets=A, max_new=1, hq=4, q=A, qs=(512, 128), shared=0, scale=0.0, out=FAR, ws=A, size=1 << 40):
    return palu.lib().palu_paged4_attn(ctypes.byref(c), tokens, offsets, max_new, hq, q, I64x2(*qs), shared, scale, out, ws, size, None)


def test_attend_refusals(palu):
    _, c = init(palu)
    for bad in (dict(tokens=0), dict(offsets=0), dict(offsets=A + 2), dict(max_new=0), dict(hq=3), dict(hq=0), dict(q=0),
                dict(q=A + 8), dict(qs=(-512, 128)), dict(qs=(512, 4)), dict(shared=5), dict(shared=-1), dict(scale=-1.0),
                dict(scale=math.inf), dict(scale=math.nan), dict(out=0), dict(out=FAR + 8), dict(out=A), dict(out=A + 256),
                dict(ws=0), dict(ws=A + 8), dict(size=10)):
        assert attend(palu, c, **bad) in (1, 2) and palu.palu_last_error(), bad
    assert attend(palu, palu.palu_paged4_cache()) == 4


def append(palu, c, tr=None, tokens=3, offsets=A, hq=4, q=A, qs=(512, 128), k=A, ks=(512, 128), v=A, vs=(512, 128), pos=None,
           q_out=FAR):
    t = palu.palu_qk_transform(**(tr or {}))
    return palu.lib().palu_paged4_append(ctypes.byref(c), ctypes.byref(t), tokens, offsets, hq, q, I64x2(*qs), k, I64x2(*ks), v,
                                         I64x2(*vs), pos, q_out, None)


def test_append_refusals(palu):
    _, c = init(palu)
    for bad in (dict(tokens=0), dict(tokens=1 << 31), dict(offsets=0), dict(offsets=A + 2), dict(hq=0), dict(q=None), dict(q_out=None),
                dict(q=A + 8), dict(k=0), dict(k=A + 4), dict(v=0), dict(ks=(512, 4)), dict(vs=(-8, 128)), dict(pos=A + 4),
                dict(q_out=A), dict(q_out=FAR + 8), dict(tr=dict(cos_sin=A, rope_dim=24, n_positions=4)),
                dict(tr=dict(cos_sin=A, rope_dim=64, n_positions=0)), dict(tr=dict(eps=-1.0)), dict(tr=dict(k_weight=A + 2)),
                dict(tokens=(1 << 31) - 1, q=None, hq=0, q_out=None, ks=(0, 0), vs=(0, 0))):
        if bad.get("tokens") == (1 << 31) - 1:                    # more blocks than a launch has
            _, wide = init(palu, hk=65536)
            assert append(palu, wide, **bad) == 2
        else:
            assert append(palu, c, **bad) in (1, 2) and palu.palu_last_error(), bad
    assert append(palu, palu.palu_paged4_cache()) == 4


def test_read_refusals(palu):
    _, c = init(palu)

    def read(tokens=3, offsets=A, starts=None, k=FAR, v=2 * FAR, cache=c):
        return palu.lib().palu_paged4_read(ctypes.byref(cache), tokens, offsets, starts, k, v, None)
    for bad in (dict(tokens=0), dict(tokens=1 << 31), dict(offsets=0), dict(offsets=A + 1), dict(starts=A + 4), dict(k=0), dict(v=0),
                dict(k=FAR + 8), dict(v=FAR), dict(v=FAR + 256), dict(k=A), dict(v=A + 7 * 10240)):
        assert read(**bad) in (1, 2) and palu.palu_last_error(), bad
    assert read(cache=palu.palu_paged4_cache()) == 4


def pool_init(palu, page=16, batch=3, width=4, n_pages=10, table=A, lengths=2 * A, held=3 * A, free=4 * A, n_free=5 * A, error=6 * A):
    p = palu.palu_page_pool()
    st = palu.lib().palu_page_pool_init(ctypes.byref(p), page, batch, width, n_pages, table, lengths, held, free, n_free, error)
    return st, p


def test_page_pool_refusals(palu):
    st, p = pool_init(palu)
    assert st == 0 and (p.page_size, p.batch, p.table_width, p.n_pages) == (16, 3, 4, 10)
    for bad in (dict(page=0), dict(page=65537), dict(batch=0), dict(batch=4097), dict(width=0), dict(width=(1 << 26) + 1),
                dict(n_pages=-1), dict(n_pages=1 << 31), dict(table=0), dict(table=A + 2), dict(lengths=0), dict(lengths=2 * A + 4),
                dict(held=0), dict(held=3 * A + 1), dict(free=0), dict(free=4 * A + 2), dict(n_free=0), dict(error=0),
                dict(error=5 * A), dict(held=A + 44), dict(free=2 * A + 20), dict(lengths=4 * A + 32)):
        st, q = pool_init(palu, **bad)
        assert st in (1, 2) and q.magic == 0 and palu.palu_last_error(), bad

    def plan(new=7 * A, tokens=5, shared=0, offsets=8 * A, positions=9 * A, slots=10 * A, pool=p):
        return palu.lib().palu_page_plan(ctypes.byref(pool), new, tokens, shared, offsets, positions, slots, None)
    for bad in (dict(new=0), dict(new=7 * A + 2), dict(tokens=-1), dict(tokens=1 << 31), dict(shared=-1), dict(shared=5),
                dict(offsets=0), dict(offsets=8 * A + 1), dict(positions=9 * A + 4), dict(slots=10 * A + 4), dict(new=3 * A + 8),
                dict(offsets=7 * A + 8), dict(positions=9 * A, slots=9 * A + 32), dict(slots=2 * A + 16), dict(offsets=A)):
        assert plan(**bad) in (1, 2) and palu.palu_last_error(), bad
    assert plan(pool=palu.palu_page_pool()) == 4


def test_rope_table_refusals(palu):
    def table(kind=0, d=64, base=1e4, factor=1.0, original=0.0, low=0.0, high=1.0, magnitude=1.0, start=0, positions=4, out=A):
        s = palu.palu_rope_scaling(kind, d, base, factor, original, low, high, magnitude)
        return palu.lib().palu_rope_table(ctypes.byref(s), start, positions, out, None)
    for bad in (dict(kind=-1), dict(kind=4), dict(d=0), dict(d=24), dict(d=144), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(kind=1, factor=0.5), dict(kind=2, factor=math.nan), dict(kind=3, factor=math.inf, original=8.0),
                dict(kind=3), dict(kind=3, original=8.0, low=-1.0), dict(kind=3, original=8.0, low=2.0, high=2.0),
                dict(kind=3, original=8.0, high=math.inf), dict(magnitude=math.nan), dict(magnitude=math.inf), dict(magnitude=1e39), dict(start=-1),
                dict(start=(1 << 40) + 1), dict(positions=-1), dict(positions=1 << 31), dict(out=0), dict(out=A + 8)):
        assert table(**bad) in (1, 2) and palu.palu_last_error(), bad
    assert table(positions=0, out=0) == 0
