// The paged cache's descriptor, and the pass that normalises and rotates
// queries and keys: into head-major tensors (palu_qk_norm_rope) or, with the
// values, into pages (palu_paged_append).
//
// The work is copying: 256-byte rows in, the same number out, a few flops a
// channel.  A CTA takes 16 consecutive tokens of a run of up to four heads, a
// half-warp a token: it reads 1 KB a token and writes 4 KB a head where the
// output is head-major.  A lane holds both members of four pairs (two 8-byte
// pieces of a row: with 16 contiguous bytes a lane the half-split pairs came by
// shuffle, and instructions, not memory, were the bound: 67 us for 16,384
// tokens of 24 + 8 heads instead of 54, 5.1 TB/s, on the device; 56 to 57 as a
// call), all four rows in flight at once; the token's angles and the norm's
// weights stay in registers for the run.  The sum of squares is
// a 4-step butterfly over the 16 lanes.  fp32 throughout, one rounding at the
// store.
#include <math.h>

#include <algorithm>

#include "qk_transform.cuh"

namespace palu {

template <bool BF16, bool INTERLEAVED, bool PAGED>
__global__ void __launch_bounds__(kAppendThreads, 5) qk_transform_kernel(const QkParams p) {
  const int tile = blockIdx.x / p.runs;
  transform_tile<BF16, INTERLEAVED, PAGED>(p, tile, blockIdx.x - tile * p.runs);
}

template <bool BF16, bool PAGED>
static palu_status launch_transform(const QkParams& p, cudaStream_t stream) {
  const long long grid = (p.rows + kAppendThreads / 16 - 1) / (kAppendThreads / 16) * p.runs;
  if (grid > 0x7fffffff) return fail(PALU_ERR_UNSUPPORTED, "too many rows for one call");
  if (p.tr.interleaved)
    qk_transform_kernel<BF16, true, PAGED><<<(unsigned)grid, kAppendThreads, 0, stream>>>(p);
  else
    qk_transform_kernel<BF16, false, PAGED><<<(unsigned)grid, kAppendThreads, 0, stream>>>(p);
  return cuda_check(cudaGetLastError(), "qk_transform_kernel launch");
}

palu_status transform_check(const palu_qk_transform* t) {
  if (!t) return fail(PALU_ERR_INVALID_ARG, "transform is NULL");
  if (((uintptr_t)t->q_weight | (uintptr_t)t->k_weight | (uintptr_t)t->cos_sin) & 15)
    return fail(PALU_ERR_INVALID_ARG, "weights and cos_sin must be 16-byte aligned");
  if (!(t->eps >= 0.f)) return fail(PALU_ERR_INVALID_ARG, "eps must not be negative");
  if (t->cos_sin) {
    if (t->rope_dim < 16 || t->rope_dim > kHeadDim || t->rope_dim % 16)
      return fail(PALU_ERR_UNSUPPORTED, "rope_dim must be a multiple of 16 in [16, 128]");
    if (t->n_positions < 1) return fail(PALU_ERR_INVALID_ARG, "n_positions must be positive");
  }
  return PALU_OK;
}

// A token-major operand: aligned, and its strides keep every row aligned.
palu_status rows_check(const char* name, const void* p, const int64_t* strides, int n) {
  if (!p || !strides) return fail(PALU_ERR_INVALID_ARG, std::string(name) + " or its strides are NULL");
  if ((uintptr_t)p & 15) return fail(PALU_ERR_INVALID_ARG, std::string(name) + " must be 16-byte aligned");
  for (int i = 0; i < n; ++i)
    if (strides[i] < 0 || strides[i] % 8)
      return fail(PALU_ERR_INVALID_ARG, std::string(name) + "'s strides must be non-negative multiples of 8 elements");
  return PALU_OK;
}

bool rows_overlap(const void* out, int64_t out_rows, const void* in, const int64_t* strides, const int64_t* extents, int n) {
  int64_t span = kHeadDim;
  for (int i = 0; i < n; ++i) span += (extents[i] - 1) * strides[i];
  const char *o = static_cast<const char*>(out), *x = static_cast<const char*>(in);
  return o < x + 2 * span && x < o + 2 * out_rows * kHeadDim;
}

palu_status paged_check(const palu_paged_cache* c) {
  if (!c) return fail(PALU_ERR_INVALID_ARG, "cache is NULL");
  if (c->magic != kPagedMagic) return fail(PALU_ERR_NOT_INITIALIZED, "paged cache is not initialised");
  return PALU_OK;
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_qk_norm_rope(const palu_qk_transform* transform, int32_t dtype, int64_t batch,
                                         int64_t tokens, int32_t q_heads, int32_t kv_heads, const void* q,
                                         const int64_t q_strides[3], const void* k, const int64_t k_strides[3],
                                         const int64_t* positions, void* q_out, void* k_out, uint32_t* error,
                                         void* stream) {
  palu_status st = transform_check(transform);
  if (st != PALU_OK) return st;
  if (dtype != PALU_TYPE_F16 && dtype != PALU_TYPE_BF16) return fail(PALU_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (batch < 1 || tokens < 1 || q_heads < 1 || kv_heads < 1 || q_heads > 65536 || kv_heads > 65536)
    return fail(PALU_ERR_INVALID_ARG, "bad shapes");
  if (batch > (1LL << 31) / tokens) return fail(PALU_ERR_UNSUPPORTED, "more than 2^31 tokens");
  if ((st = rows_check("q", q, q_strides, 3)) != PALU_OK || (st = rows_check("k", k, k_strides, 3)) != PALU_OK) return st;
  if (!q_out || !k_out || (((uintptr_t)q_out | (uintptr_t)k_out) & 15))
    return fail(PALU_ERR_INVALID_ARG, "q_out and k_out must be 16-byte aligned");
  const int64_t qe[3] = {batch, tokens, q_heads}, ke[3] = {batch, tokens, kv_heads};
  const int64_t q_rows = batch * tokens * q_heads, k_rows = batch * tokens * kv_heads, row_stride = kHeadDim;
  if (rows_overlap(q_out, q_rows, q, q_strides, qe, 3) || rows_overlap(q_out, q_rows, k, k_strides, ke, 3) ||
      rows_overlap(k_out, k_rows, q, q_strides, qe, 3) || rows_overlap(k_out, k_rows, k, k_strides, ke, 3) ||
      rows_overlap(q_out, q_rows, k_out, &row_stride, &k_rows, 1))
    return fail(PALU_ERR_INVALID_ARG, "an output overlaps an input or the other output");
  if (transform->cos_sin && (!positions || ((uintptr_t)positions & 7)))
    return fail(PALU_ERR_INVALID_ARG, "positions must be given, 8-byte aligned, with a table");
  QkParams p = {};
  p.tr = *transform;
  if (!p.tr.cos_sin) p.tr.rope_dim = 0;  // no pairs
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.qs0 = q_strides[0], p.qs1 = q_strides[1], p.qs2 = q_strides[2];
  p.ks0 = k_strides[0], p.ks1 = k_strides[1], p.ks2 = k_strides[2];
  p.positions = reinterpret_cast<const long long*>(positions);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.error = error;
  p.rows = batch * tokens;
  p.tokens = tokens;
  p.hq = q_heads;
  p.hk = kv_heads;
  p.q_runs = (q_heads + kRunHeads - 1) / kRunHeads;
  p.k_runs = (kv_heads + kRunHeads - 1) / kRunHeads;
  p.runs = p.q_runs + p.k_runs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == PALU_TYPE_BF16 ? launch_transform<true, false>(p, s) : launch_transform<false, false>(p, s);
}

extern "C" palu_status palu_paged_cache_init(palu_paged_cache* cache, int32_t dtype, int32_t kv_heads,
                                             int32_t page_size, int64_t n_pages, void* k_pages,
                                             const int64_t k_strides[3], void* v_pages, const int64_t v_strides[3],
                                             const int32_t* page_table, int64_t batch, int64_t table_width,
                                             const int64_t* lengths, uint32_t* error) {
  if (!cache) return fail(PALU_ERR_INVALID_ARG, "cache is NULL");
  cache->magic = 0;
  if (dtype != PALU_TYPE_F16 && dtype != PALU_TYPE_BF16) return fail(PALU_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(PALU_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (kv_heads < 1 || kv_heads > 65536 || n_pages < 1 || n_pages > 0x7fffffff)
    return fail(PALU_ERR_INVALID_ARG, "bad head or page count");
  if (batch < 1 || table_width < 1) return fail(PALU_ERR_INVALID_ARG, "batch and table_width must be positive");
  if (batch > kMaxPagedBatch) return fail(PALU_ERR_UNSUPPORTED, "at most 4096 sequences");
  // places are 32-bit numbers inside the attention kernels
  if (table_width > (1LL << 30) / page_size) return fail(PALU_ERR_UNSUPPORTED, "at most 2^30 tokens a sequence");
  palu_status st;
  if ((st = rows_check("k_pages", k_pages, k_strides, 3)) != PALU_OK ||
      (st = rows_check("v_pages", v_pages, v_strides, 3)) != PALU_OK)
    return st;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] < 8 || v_strides[i] < 8 || k_strides[i] >= (1LL << 38) || v_strides[i] >= (1LL << 38))
      return fail(PALU_ERR_INVALID_ARG, "page strides must be positive (and less than 2^38 elements)");
  if (!page_table || !lengths || !error) return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if (((uintptr_t)page_table | (uintptr_t)error) & 3 || (uintptr_t)lengths & 7)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  cache->dtype = dtype;
  cache->kv_heads = kv_heads;
  cache->page_size = page_size;
  cache->batch = (int32_t)batch;
  cache->table_width = (int32_t)table_width;
  cache->n_pages = n_pages;
  cache->k_pages = k_pages;
  cache->v_pages = v_pages;
  for (int i = 0; i < 3; ++i) {
    cache->k_strides[i] = k_strides[i];
    cache->v_strides[i] = v_strides[i];
  }
  cache->page_table = page_table;
  cache->lengths = lengths;
  cache->error = error;
  cache->magic = kPagedMagic;
  return PALU_OK;
}

extern "C" palu_status palu_paged_append(const palu_paged_cache* cache, const palu_qk_transform* transform,
                                         int64_t tokens, const int32_t* offsets, int32_t q_heads, const void* q,
                                         const int64_t q_strides[2], const void* k, const int64_t k_strides[2],
                                         const void* v, const int64_t v_strides[2], const int64_t* positions,
                                         void* q_out, void* stream) {
  palu_status st = paged_check(cache);
  if (st != PALU_OK || (st = transform_check(transform)) != PALU_OK) return st;
  if (tokens < 1 || tokens > 0x7fffffff) return fail(PALU_ERR_INVALID_ARG, "tokens must be in [1, 2^31)");
  if (q_heads < 0 || q_heads > 65536 || (q_heads > 0) != (q != nullptr) || (q_heads > 0) != (q_out != nullptr))
    return fail(PALU_ERR_INVALID_ARG, "q, q_out and q_heads come together");
  if (!offsets || ((uintptr_t)offsets & 3)) return fail(PALU_ERR_INVALID_ARG, "offsets must be given, 4-byte aligned");
  if (q && (st = rows_check("q", q, q_strides, 2)) != PALU_OK) return st;
  if ((st = rows_check("k", k, k_strides, 2)) != PALU_OK || (st = rows_check("v", v, v_strides, 2)) != PALU_OK) return st;
  if ((uintptr_t)q_out & 15) return fail(PALU_ERR_INVALID_ARG, "q_out must be 16-byte aligned");
  if ((uintptr_t)positions & 7) return fail(PALU_ERR_INVALID_ARG, "positions must be 8-byte aligned");
  const int64_t qe[2] = {tokens, q_heads}, ke[2] = {tokens, cache->kv_heads};
  if (q && (rows_overlap(q_out, tokens * q_heads, q, q_strides, qe, 2) || rows_overlap(q_out, tokens * q_heads, k, k_strides, ke, 2) ||
            rows_overlap(q_out, tokens * q_heads, v, v_strides, ke, 2)))
    return fail(PALU_ERR_INVALID_ARG, "q_out overlaps an input");
  QkParams p = {};
  p.tr = *transform;
  if (!p.tr.cos_sin) p.tr.rope_dim = 0;  // no pairs
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  if (q) p.qs1 = q_strides[0], p.qs2 = q_strides[1];
  p.ks1 = k_strides[0], p.ks2 = k_strides[1];
  p.vs1 = v_strides[0], p.vs2 = v_strides[1];
  p.positions = reinterpret_cast<const long long*>(positions);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.error = cache->error;
  p.rows = tokens;
  p.tokens = tokens;
  p.hq = q_heads;
  p.hk = cache->kv_heads;
  p.q_runs = (q_heads + kRunHeads - 1) / kRunHeads;
  p.k_runs = (cache->kv_heads + kRunHeads - 1) / kRunHeads;
  p.runs = p.q_runs + 2 * p.k_runs;
  p.offsets = offsets;
  p.c = paged_view(cache);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->dtype == PALU_TYPE_BF16 ? launch_transform<true, true>(p, s) : launch_transform<false, true>(p, s);
}

extern "C" palu_status palu_paged_sync(const palu_paged_cache* cache, uint32_t* device_error, void* stream) {
  palu_status st = paged_check(cache);
  if (st != PALU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t e = 0;
  st = cuda_check(cudaMemcpyAsync(&e, cache->error, sizeof(e), cudaMemcpyDeviceToHost, s), "cudaMemcpyAsync(error word)");
  if (st != PALU_OK || (st = cuda_check(cudaStreamSynchronize(s), "cudaStreamSynchronize")) != PALU_OK) return st;
  if (device_error) *device_error = e;
  if (!e) return PALU_OK;
  if ((st = cuda_check(cudaMemsetAsync(cache->error, 0, sizeof(e), s), "cudaMemsetAsync(error word)")) != PALU_OK) return st;
  std::string msg = "device error word " + std::to_string(e) + ":";
  if (e & PALU_DEVERR_CAPACITY) msg += " a length past the page table;";
  if (e & PALU_DEVERR_PAGE) msg += " a page id outside the pool;";
  if (e & PALU_DEVERR_SPAN) msg += " offsets out of order, or more new tokens than the sequence or the call has;";
  if (e & PALU_DEVERR_POSITION) msg += " a position outside the rotation table;";
  if (e & PALU_DEVERR_TIMEOUT) msg += " a bounded wait ran out;";
  return fail(PALU_ERR_DEVICE, msg);
}
