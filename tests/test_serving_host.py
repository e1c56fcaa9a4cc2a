"""Host side of include/paged.h and include/draft.h without a GPU: the structs
match the headers, and every argument that a call can refuse is refused with a
status and a message before anything is launched."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from tests.conftest import ROOT
from tests.test_abi import palu  # noqa: F401  (fixture)

I64x3, I64x2 = ctypes.c_int64 * 3, ctypes.c_int64 * 2
A = 1 << 20            # an aligned address that is never read


def test_struct_layouts_match_the_header(palu):
    prog = r'''
#include <stdio.h>
#include <stddef.h>
#include "paged.h"
#include "draft.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(palu_qk_transform), offsetof(palu_qk_transform, eps), sizeof(palu_paged_cache),
         offsetof(palu_paged_cache, k_strides), offsetof(palu_paged_cache, page_table), offsetof(palu_paged_cache, error));
  return 0;
}'''
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(src, "w") as f:
            f.write(prog)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        vals = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    t, c = palu.palu_qk_transform, palu.palu_paged_cache
    packed = palu._pack_transform(1, 2, 3, 4, 5, 6, 7.5, 0)
    x = t.from_buffer_copy(packed)
    assert len(packed) == vals[0] and (x.q_weight, x.k_weight, x.cos_sin, x.n_positions, x.rope_dim, x.interleaved, x.eps) == \
        (1, 2, 3, 4, 5, 6, 7.5)
    assert vals == [ctypes.sizeof(t), t.eps.offset, ctypes.sizeof(c), c.k_strides.offset, c.page_table.offset, c.error.offset]


def init(palu, dtype=0, hk=2, page=16, n_pages=8, k=A, ks=(4096, 2048, 128), v=A, vs=(4096, 2048, 128), table=A, batch=3,
         width=4, lengths=A, error=A):
    c = palu.palu_paged_cache()
    st = palu.lib().palu_paged_cache_init(ctypes.byref(c), dtype, hk, page, n_pages, k, I64x3(*ks), v, I64x3(*vs), table, batch,
                                          width, lengths, error)
    return st, c


def test_cache_init(palu):
    st, c = init(palu)
    assert st == 0 and (c.kv_heads, c.page_size, c.batch, c.table_width, c.n_pages) == (2, 16, 3, 4, 8)
    for bad in (dict(dtype=2), dict(hk=0), dict(page=24), dict(page=256), dict(page=0), dict(n_pages=0), dict(n_pages=1 << 31),
                dict(k=0), dict(k=A + 8), dict(ks=(4096, 2048, 4)), dict(ks=(-4096, 2048, 128)), dict(ks=(0, 2048, 128)),
                dict(vs=(4096, 2044, 128)), dict(vs=(1 << 40, 2048, 128)), dict(v=0), dict(table=0), dict(table=A + 2),
                dict(batch=0), dict(batch=4097), dict(width=0), dict(width=(1 << 26) + 1), dict(lengths=0), dict(lengths=A + 4),
                dict(error=0), dict(error=A + 1)):
        st, c = init(palu, **bad)
        assert st in (1, 2) and c.magic == 0 and palu.palu_last_error(), bad


def test_workspace_size(palu):
    _, c = init(palu)
    n = ctypes.c_size_t()
    size = lambda *a: palu.lib().palu_paged_attn_workspace_size(ctypes.byref(c), *a, ctypes.byref(n))
    assert size(3, 4, 1, 0) == 0 and n.value > 0 and n.value % 256 == 0
    plain = n.value
    assert size(3, 4, 1, 2) == 0 and n.value > plain
    for bad in ((0, 4, 1, 0), (3, 0, 1, 0), (3, 3, 1, 0), (3, 4, 0, 0), (3, 4, 1, 5), (3, 4, 1, -1), (3, 130, 1, 0), (1 << 30, 4, 1, 0)):
        assert size(*bad) in (1, 2), bad
    assert palu.lib().palu_paged_attn_workspace_size(ctypes.byref(palu.palu_paged_cache()), 3, 4, 1, 0, ctypes.byref(n)) == 4


@pytest.mark.parametrize("width", [4, 40])
def test_a_workspace_serves_smaller_calls(palu, width):
    _, c = init(palu, width=width, batch=30)
    n = ctypes.c_size_t()

    def size(tokens, new, shared):
        assert palu.lib().palu_paged_attn_workspace_size(ctypes.byref(c), tokens, 14, new, shared, ctypes.byref(n)) == 0
        return n.value
    sizes = [(t, m) for t in (1, 2, 3, 30, 100, 300) for m in (1, 2, 3, 10, 100)]
    for t, m in sizes:
        shared = {size(t, m, s) for s in range(1, width + 1)}
        assert len(shared) == 1 and size(t, m, 0) <= shared.pop()
        for t1, m1 in sizes:
            if t1 <= t and m1 <= m:
                assert all(size(t1, m1, s) <= size(t, m, s) for s in (0, 1, width // 2, width))


def transform(palu, **kw):
    t = palu.palu_qk_transform()
    for k, v in dict(dict(cos_sin=A, n_positions=100, rope_dim=64), **kw).items():
        setattr(t, k, v)
    return t


def test_qk_norm_rope_refusals(palu):
    def call(t=None, dtype=0, b=2, n=3, hq=4, hk=2, q=A, qs=(1536, 512, 128), k=A, ks=(768, 256, 128), pos=A, qo=2 * A, ko=3 * A):
        t = transform(palu) if t is None else t
        return palu.lib().palu_qk_norm_rope(ctypes.byref(t), dtype, b, n, hq, hk, q, I64x3(*qs), k, I64x3(*ks), pos, qo, ko, None,
                                            None)
    for bad in (dict(t=transform(palu, rope_dim=8)), dict(t=transform(palu, rope_dim=144)), dict(t=transform(palu, rope_dim=24)),
                dict(t=transform(palu, n_positions=0)), dict(t=transform(palu, eps=-1.0)), dict(t=transform(palu, eps=float("nan"))),
                dict(t=transform(palu, q_weight=A + 2)), dict(t=transform(palu, cos_sin=A + 4)), dict(dtype=3), dict(b=0),
                dict(n=0), dict(hq=0), dict(hk=0), dict(b=1 << 20, n=1 << 20), dict(q=0), dict(q=A + 2), dict(qs=(1536, 512, 4)),
                dict(qs=(-8, 512, 128)), dict(k=0), dict(pos=0), dict(pos=A + 4), dict(qo=0), dict(ko=3 * A + 8), dict(qo=A), dict(ko=A + 256)):
        assert call(**bad) in (1, 2) and palu.palu_last_error(), bad


def test_append_and_attend_refusals(palu):
    _, c = init(palu)
    t = transform(palu)

    def append(c=c, t=t, n=3, off=A, hq=4, q=A, qs=(512, 128), k=A, ks=(256, 128), v=A, vs=(256, 128), pos=None, qo=2 * A):
        return palu.lib().palu_paged_append(ctypes.byref(c), ctypes.byref(t), n, off, hq, q, I64x2(*qs), k, I64x2(*ks), v,
                                            I64x2(*vs), pos, qo, None)
    for bad in (dict(c=palu.palu_paged_cache()), dict(n=0), dict(n=1 << 31), dict(off=None), dict(off=A + 2), dict(hq=0),
                dict(q=None), dict(qo=None), dict(q=A + 2), dict(qs=(512, 4)), dict(k=None), dict(ks=(-256, 128)), dict(v=None),
                dict(v=A + 2), dict(pos=A + 4), dict(qo=2 * A + 8), dict(qo=A), dict(k=2 * A), dict(t=transform(palu, rope_dim=40))):
        assert append(**bad) in (1, 2, 4), bad

    def attend(c=c, n=3, off=A, new=1, hq=4, q=A, qs=(512, 128), shared=0, scale=0.0, out=2 * A, ws=A, wb=1 << 30):
        return palu.lib().palu_paged_attn(ctypes.byref(c), n, off, new, hq, q, I64x2(*qs), shared, scale, out, ws, wb, None)
    for bad in (dict(c=palu.palu_paged_cache()), dict(n=0), dict(off=None), dict(off=A + 1), dict(new=0), dict(hq=3), dict(q=None),
                dict(q=A + 8), dict(qs=(512, 4)), dict(qs=(-512, 128)), dict(shared=5), dict(shared=-1), dict(scale=-1.0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None), dict(out=A), dict(out=A + 16), dict(out=2 * A + 2), dict(ws=None), dict(wb=100)):
        assert attend(**bad) in (1, 2, 4), bad


def test_draft_verify_refusals(palu):
    def call(b=2, k=3, V=50, t=A, ts=(200, 50), d=A, ds=(150, 50), x=A, n=None, au=A, su=A, le=None, tok=2 * A, kept=A, nl=None):
        return palu.lib().palu_draft_verify(b, k, V, t, I64x2(*ts), d, I64x2(*ds), x, n, au, su, le, tok, kept, nl, None)
    for bad in (dict(b=0), dict(b=1 << 25), dict(k=0), dict(k=257), dict(V=0), dict(V=1 << 31), dict(t=None), dict(t=A + 2),
                dict(ts=(-1, 50)), dict(ds=(150, -1)), dict(x=None), dict(x=A + 4), dict(au=None), dict(su=None), dict(tok=None),
                dict(tok=A), dict(kept=None), dict(le=A), dict(nl=A), dict(n=A + 1)):
        assert call(**bad) in (1, 2) and palu.palu_last_error(), bad


def test_outputs_that_overlap_are_refused(palu):
    t = transform(palu)
    n = 2 * 3 * 2 * 128 * 2                      # bytes of k_out

    def rope(qo, ko):
        return palu.lib().palu_qk_norm_rope(ctypes.byref(t), 0, 2, 3, 4, 2, A, I64x3(1536, 512, 128), A, I64x3(768, 256, 128), A, qo,
                                            ko, None, None)
    for qo, ko in ((2 * A, 2 * A), (2 * A, 2 * A + n), (2 * A + n - 256, 2 * A)):
        assert rope(qo, ko) == 1 and b"overlap" in palu.lib().palu_last_error()

    # tokens [2, 4] (64 bytes) against drafts [2, 3] (48), n_drafts (8), accept_u (24), sample_u (8), lengths (16)
    def verify(tok, x=2 * A, n=3 * A, au=4 * A, su=5 * A, le=6 * A):
        return palu.lib().palu_draft_verify(2, 3, 50, A, I64x2(200, 50), A, I64x2(150, 50), x, n, au, su, le, tok, A, A, None)
    for at, size in ((2 * A, 48), (3 * A, 8), (4 * A, 24), (5 * A, 8), (6 * A, 16)):
        for tok in (at, at + size - 8, at - 56):
            assert verify(tok) == 1 and b"overlap" in palu.lib().palu_last_error(), (at, tok)


def test_a_workspace_serves_calls_that_share_and_calls_that_do_not(palu):
    """Whether shared pages are read once depends on the sizes: the size of a workspace must not fall where it changes."""
    _, c = init(palu, hk=64, ks=(1 << 18, 2048, 128), vs=(1 << 18, 2048, 128), width=200, batch=30)
    n = ctypes.c_size_t()

    def size(tokens, new, shared):
        assert palu.lib().palu_paged_attn_workspace_size(ctypes.byref(c), tokens, 128, new, shared, ctypes.byref(n)) == 0
        return n.value
    for new in (1, 3, 9, 200, 100000):
        for shared in (0, 1, 8, 9, 100, 200):
            sizes = [size(t, new, shared) for t in (1, 2, 29, 30, 31, 60, 90, 270, 300, 900, 1000, 2000, 5000, 6000, 10000, 100000)]
            assert sizes == sorted(sizes)
    for t in (30, 300, 5000, 100000):
        for shared in (0, 1, 8, 9, 100, 200):
            sizes = [size(t, new, shared) for new in (1, 2, 3, 8, 9, 10, 200, 100000)]
            assert sizes == sorted(sizes)
        assert len({size(t, 9, s) for s in (1, 7, 8, 9, 40, 200)}) == 1
    assert size(100000, 9, 8) < 100000 * 128 * 520         # no record of every row where they are never shared
