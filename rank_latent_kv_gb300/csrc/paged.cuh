// Shared by the paged-cache translation units: the cache as kernels see it,
// and which sequence and place a new token has.
#pragma once

#include "paged.h"
#include "palu_internal.cuh"

namespace palu {

constexpr int32_t kPagedMagic = 0x50414745;  // "PAGE"
constexpr int kMaxPagedBatch = 4096;
constexpr int kMaxPagedGq = 64;

struct PagedView {
  uint16_t *k, *v;                       // 16-bit elements of either type
  long long ks0, ks1, ks2, vs0, vs1, vs2;  // page, head, token strides in elements
  const int* table;
  const long long* lengths;
  unsigned int* error;
  long long n_pages;
  int batch, width, kv_heads, page, page_shift;
};

inline PagedView paged_view(const palu_paged_cache* c) {
  PagedView v;
  v.k = static_cast<uint16_t*>(c->k_pages);
  v.v = static_cast<uint16_t*>(c->v_pages);
  v.ks0 = c->k_strides[0];
  v.ks1 = c->k_strides[1];
  v.ks2 = c->k_strides[2];
  v.vs0 = c->v_strides[0];
  v.vs1 = c->v_strides[1];
  v.vs2 = c->v_strides[2];
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

// PALU_OK, or why the descriptor cannot be used.
palu_status paged_check(const palu_paged_cache* c);

// Whether the contiguous 16-bit rows of an output share memory with a strided
// operand of these extents (by their address ranges).
bool rows_overlap(const void* out, int64_t out_rows, const void* in, const int64_t* strides, const int64_t* extents, int n);

// Largest b in [0, batch) with offsets[b] <= row, searched by 16 lanes at
// once (`lane` 0..15; `mask` their lanes of the warp): each step cuts the range
// to a sixteenth, so the dependent loads are one for up to 16 sequences and
// three for 4096.  Any contents of offsets give an answer in [0, batch).
__device__ __forceinline__ int find_sequence(const int* offsets, int batch, int row, int lane, unsigned mask) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 15) >> 4;
    const int at = lane * step;  // probe the start of this lane's part
    const bool le = at < n && (at == 0 || __ldg(offsets + lo + at) <= row);
    unsigned hits = __ballot_sync(mask, le) & mask;
    hits = mask >> 16 ? hits >> 16 : hits;  // mask is one half of the warp
    const int part = 31 - __clz(hits & 0xffffu);
    lo += part * step;
    n = min(step, n - part * step);
  }
  return lo;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF16) return make_float2(bf16_lo_to_f32(v), bf16_hi_to_f32(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

}  // namespace palu
