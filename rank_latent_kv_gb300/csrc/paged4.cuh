// Shared by the translation units of the 4-bit paged cache: where a block's
// fields lie, and which block of which sequence a CTA has.
#pragma once

#include "paged.cuh"
#include "paged4.h"

namespace palu {

constexpr int32_t kPaged4Magic = 0x50473442;  // "PG4B"
constexpr int kBlock4 = PALU_PAGED4_BLOCK;    // bytes of 16 tokens
constexpr int kKeyScales4 = 1024, kValueCodes4 = 1280, kValueScales4 = 2304;

// As kernels see it: k is the pool, ks0 and ks1 its strides in bytes.
inline PagedView paged4_view(const palu_paged4_cache* c) {
  PagedView v = {};
  v.k = static_cast<uint16_t*>(c->pages);
  v.ks0 = c->strides[0];
  v.ks1 = c->strides[1];
  v.table = c->page_table;
  v.lengths = reinterpret_cast<const long long*>(c->lengths);
  v.error = c->error;
  v.n_pages = c->n_pages;
  v.batch = c->batch;
  v.width = c->table_width;
  v.kv_heads = c->kv_heads;
  v.page = c->page_size;
  v.page_shift = __builtin_ctz(c->page_size);
  return v;
}

palu_status paged4_check(const palu_paged4_cache* c);

// The page of a head, in a pool of blocks.
__device__ __forceinline__ uint8_t* page4(const PagedView& c, int page, int head) {
  return reinterpret_cast<uint8_t*>(c.k) + (long long)page * c.ks0 + (long long)head * c.ks1;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Queries enter fp16 products times 2^e, e such that the row's largest value
// `big` comes to 2^13 .. 2^14 (rows of zeros or of infinities: as they are), and
// the factor that takes the products back to log2: not 0, whatever the scale, so
// that a masked score of -infinity stays one, and not infinite (queries above 2^118
// give one key all the weight, by whatever factor).
__device__ __forceinline__ int query_shift(float big) {
  const int ex = (int)(__float_as_uint(big) >> 23);
  return ex == 0 || ex == 255 ? 0 : max(min(13 + 127 - ex, 100), -113);
}
__device__ __forceinline__ float query_factor(int e, float scale_log2) {
  return fminf(fmaxf(__uint_as_float((uint32_t)(127 - e) << 23) * scale_log2, 0x1p-120f), 3e38f);
}

// Work on whole blocks without a scan over the sequences: n rows touch at most
// n / 16 + 2 blocks wherever they begin, so sequence b has the CTAs from
// offsets[b] / 16 + 2 b on, and there are tokens / 16 + 2 batch of them.
__device__ __forceinline__ int first_block_cta(const int* offsets, int b) { return (__ldg(offsets + b) >> 4) + 2 * b; }

// The sequence of CTA x, searched as find_sequence does.
__device__ __forceinline__ int find_block(const int* offsets, int batch, int x, int lane, unsigned mask) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 15) >> 4, at = lane * step;
    const bool le = at < n && (at == 0 || first_block_cta(offsets, lo + at) <= x);
    unsigned hits = __ballot_sync(mask, le) & mask;
    hits = mask >> 16 ? hits >> 16 : hits;
    const int part = 31 - __clz(hits & 0xffffu);
    lo += part * step;
    n = min(step, n - part * step);
  }
  return lo;
}

// What a CTA's 16 half-warps do: token `place` of sequence b, in row `row` of
// the call, where `live`; all in one block.
struct BlockWork {
  int place, row;
  bool live;
  int page, in_page;  // the block's page, and its place there
};

// Which block CTA x has (uniform: false for all threads or none).  The tokens are
// sequence b's from starts[b] on (its last ones without starts).  Errors of a
// sequence are found by CTA x = b, whatever else it has, if `tell`.
__device__ __forceinline__ bool block_work(const PagedView& c, const int* offsets, const long long* starts, long long rows, int x,
                                           bool tell, BlockWork* w) {
  const int lane = threadIdx.x & 15;
  auto span = [&](int b, int* o0, int* n, long long* first, long long* len) -> unsigned {
    *o0 = __ldg(offsets + b);
    const int o1 = __ldg(offsets + b + 1);
    *n = o1 - *o0;
    *len = __ldg(c.lengths + b);
    *first = starts ? __ldg(starts + b) : *len - *n;
    if (*o0 < 0 || o1 < *o0 || o1 > rows || *first < 0 || *first > *len - *n) return PALU_DEVERR_SPAN;
    return *len > (long long)c.width * c.page ? PALU_DEVERR_CAPACITY : 0u;
  };
  int o0, n;
  long long first, len;
  if (tell && x < c.batch && threadIdx.x == 0) {
    unsigned bad = span(x, &o0, &n, &first, &len);
    if (n == 0 && o0 >= 0 && o0 <= rows) bad = 0;  // no tokens: no matter what its length is
    if (x == 0 && o0 != 0) bad |= PALU_DEVERR_SPAN;
    if (bad) atomicOr(c.error, bad);
  }
  const int b = find_block(offsets, c.batch, x, lane, (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu);
  if (span(b, &o0, &n, &first, &len)) return false;
  const int j = x - ((o0 >> 4) + 2 * b);
  const long long blk = (first >> 4) + j, at = blk * 16;  // the block's first place
  if (n == 0 || j < 0 || at >= first + n) return false;
  w->place = (int)at + (threadIdx.x >> 4);
  w->live = w->place >= first && w->place < first + n;
  w->row = o0 + (int)(w->place - first);
  w->page = __ldg(c.table + (long long)b * c.width + (at >> c.page_shift));
  w->in_page = ((int)at & (c.page - 1)) >> 4;
  return true;
}

// Its block of head 0, or nullptr and an error bit (uniform); to be asked for when the rows' loads are under way.
__device__ __forceinline__ uint8_t* block_of_work(const PagedView& c, const BlockWork& w) {
  if (w.page < 0 || w.page >= c.n_pages) {
    if (threadIdx.x == 0) atomicOr(c.error, PALU_DEVERR_PAGE);
    return nullptr;
  }
  return page4(c, w.page, 0) + w.in_page * kBlock4;
}

}  // namespace palu
