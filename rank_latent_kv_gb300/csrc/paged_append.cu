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

#include "paged.cuh"

namespace palu {

constexpr int kRunHeads = 4;       // heads a half-warp takes
constexpr int kAppendThreads = 256;

struct QkParams {
  palu_qk_transform tr;
  const uint16_t *q, *k, *v;
  long long qs0, qs1, qs2, ks0, ks1, ks2, vs1, vs2;  // batch, token, head strides in elements
  const long long* positions;
  uint16_t *q_out, *k_out;
  unsigned int* error;
  long long rows;      // tokens of all sequences
  long long tokens;    // tokens of a sequence (dense form)
  int hq, hk, q_runs, k_runs, runs;
  const int* offsets;  // paged form
  PagedView c;
};

// A row's two pieces of four channels a lane: the norm (by w, where there is
// one), then the rotation of the lane's four pairs: (x0, x4) .. (x3, x7), or
// (x0, x1) .. (x6, x7) when interleaved.
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void transform_row(uint2& lo, uint2& hi, bool norm, const float (&w)[8], bool turn,
                                              const float4& co, const float4& si, float eps, unsigned mask) {
  float x[8];
  const uint32_t raw[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(raw[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  if (norm) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
    for (int m = 8; m; m >>= 1) s += __shfl_xor_sync(mask, s, m);
    const float r = rsqrtf(s * (1.f / kHeadDim) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (turn) {
    const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = INTERLEAVED ? 2 * i : i, k = INTERLEAVED ? 2 * i + 1 : i + 4;
      const float a = x[j], b = x[k];
      x[j] = a * c[i] - b * s[i];
      x[k] = b * c[i] + a * s[i];
    }
  }
  lo = make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
  hi = make_uint2(pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}

template <bool BF16, bool INTERLEAVED, bool PAGED>
__global__ void __launch_bounds__(kAppendThreads, 5) qk_transform_kernel(const QkParams p) {
  const int lane = threadIdx.x & 15;
  const unsigned mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  const int tile = blockIdx.x / p.runs, run = blockIdx.x - tile * p.runs;
  const long long row = (long long)tile * (kAppendThreads / 16) + (threadIdx.x >> 4);
  if (row >= p.rows) return;
  // which heads: queries, keys, then (paged form) values
  const int kind = run < p.q_runs ? 0 : run < p.q_runs + p.k_runs ? 1 : 2;
  const int h0 = (kind == 0 ? run : kind == 1 ? run - p.q_runs : run - p.q_runs - p.k_runs) * kRunHeads;
  const int nh = min(kRunHeads, (kind == 0 ? p.hq : p.hk) - h0);
  const long long bi = PAGED ? 0 : row / p.tokens, ti = PAGED ? row : row - bi * p.tokens;
  const uint16_t* src = kind == 0   ? p.q + bi * p.qs0 + ti * p.qs1 + (long long)h0 * p.qs2
                        : kind == 1 ? p.k + bi * p.ks0 + ti * p.ks1 + (long long)h0 * p.ks2
                                    : p.v + ti * p.vs1 + (long long)h0 * p.vs2;
  const long long hs = kind == 0 ? p.qs2 : kind == 1 ? p.ks2 : p.vs2;
  // the lane's channels: ca .. ca+3 and cb .. cb+3
  const bool pairs = lane < (p.tr.rope_dim >> 3);
  const int ca = !INTERLEAVED && pairs ? 4 * lane : 8 * lane;
  const int cb = !INTERLEAVED && pairs ? (p.tr.rope_dim >> 1) + 4 * lane : 8 * lane + 4;
  uint2 lo[kRunHeads], hi[kRunHeads];
#pragma unroll
  for (int i = 0; i < kRunHeads; ++i)
    if (i < nh) {
      lo[i] = __ldg(reinterpret_cast<const uint2*>(src + i * hs + ca));
      hi[i] = __ldg(reinterpret_cast<const uint2*>(src + i * hs + cb));
    }

  // the token's place, and whether it may be written
  long long pos = 0, page = 0;
  int slot = 0;
  unsigned bad = 0;
  if (PAGED) {
    const int b = find_sequence(p.offsets, p.c.batch, (int)row, lane, mask);
    const int o0 = __ldg(p.offsets + b), o1 = __ldg(p.offsets + b + 1);
    if (row >= __ldg(p.offsets + p.c.batch)) return;  // behind the last sequence
    const long long len = __ldg(p.c.lengths + b);
    if (o0 < 0 || row < o0 || row >= o1 || o1 > p.rows || len < o1 - o0)
      bad = PALU_DEVERR_SPAN;
    else if (len > (long long)p.c.width * p.c.page)
      bad = PALU_DEVERR_CAPACITY;
    else {
      pos = len - o1 + row;
      slot = (int)(pos & (p.c.page - 1));
      page = __ldg(p.c.table + (long long)b * p.c.width + (pos >> p.c.page_shift));
      if (page < 0 || page >= p.c.n_pages) bad = PALU_DEVERR_PAGE;
    }
  }
  const bool turn = kind < 2 && pairs;
  float4 co = {}, si = {};
  if (p.tr.cos_sin != nullptr) {
    if (p.positions) pos = __ldg(p.positions + row);
    if (!bad && (pos < 0 || pos >= p.tr.n_positions)) bad = PALU_DEVERR_POSITION;
    if (!bad && turn) {
      const float* cs = p.tr.cos_sin + pos * p.tr.rope_dim + 4 * lane;
      co = __ldg(reinterpret_cast<const float4*>(cs));
      si = __ldg(reinterpret_cast<const float4*>(cs + (p.tr.rope_dim >> 1)));
    }
  }
  if (bad && lane == 0 && p.error) atomicOr(p.error, bad);
  if (bad && PAGED && kind > 0) return;  // nothing of it is appended

  const uint16_t* wsrc = static_cast<const uint16_t*>(kind == 0 ? p.tr.q_weight : kind == 1 ? p.tr.k_weight : nullptr);
  float w[8] = {};
  if (wsrc) {
    const uint2 wl = __ldg(reinterpret_cast<const uint2*>(wsrc + ca)), wh = __ldg(reinterpret_cast<const uint2*>(wsrc + cb));
    const uint32_t raw[4] = {wl.x, wl.y, wh.x, wh.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(raw[i]);
      w[2 * i] = f.x;
      w[2 * i + 1] = f.y;
    }
  }
  uint16_t* dst;
  long long ds;  // between heads
  if (PAGED) {
    if (kind == 0) {
      dst = p.q_out + (row * p.hq + h0) * kHeadDim;
      ds = kHeadDim;
    } else if (kind == 1) {
      dst = p.c.k + page * p.c.ks0 + h0 * p.c.ks1 + slot * p.c.ks2;
      ds = p.c.ks1;
    } else {
      dst = p.c.v + page * p.c.vs0 + h0 * p.c.vs1 + slot * p.c.vs2;
      ds = p.c.vs1;
    }
  } else {
    dst = (kind == 0 ? p.q_out : p.k_out) + ((bi * (kind == 0 ? p.hq : p.hk) + h0) * p.tokens + ti) * kHeadDim;
    ds = p.tokens * kHeadDim;
  }
  const uint32_t nan2 = 0x7fff7fffu;  // a NaN in either type
#pragma unroll
  for (int i = 0; i < kRunHeads; ++i) {
    if (i < nh) {  // the same for all 16 lanes
      if (bad)
        lo[i] = hi[i] = make_uint2(nan2, nan2);
      else if (kind < 2)
        transform_row<BF16, INTERLEAVED>(lo[i], hi[i], wsrc != nullptr, w, turn, co, si, p.tr.eps, mask);
      *reinterpret_cast<uint2*>(dst + i * ds + ca) = lo[i];
      *reinterpret_cast<uint2*>(dst + i * ds + cb) = hi[i];
    }
  }
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

static palu_status transform_check(const palu_qk_transform* t) {
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
static palu_status rows_check(const char* name, const void* p, const int64_t* strides, int n) {
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
