// The paged attention's host side, and the joining of partial results.
#include <math.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "splitk_attend.cuh"

namespace palu {

// ---- joining.  Eight warps a CTA: all on one row, every eighth part each, where
// rows are few and may have up to a part an SM (a single long sequence); else
// a warp a row, unless a row turns out to have many parts after all.  Lanes hold
// four channels.  Parts are joined in a fixed order: the result repeats bit
// for bit.
constexpr int kJoinWarps = 8;
constexpr int kJoinFew = 64;       // parts up to which a warp joins alone
constexpr int kJoinRows = 256;     // rows up to which each gets a CTA

struct JoinScratch {
  float o[kJoinWarps][kHeadDim];
  float2 ml[kJoinWarps];
};

struct Joined {
  float M, L, o[4];
};

// Parts k0, k0 + step, ... < n of a row; part(k, &ml, &acc) says where part k lies.
template <class F>
__device__ __forceinline__ Joined join_parts(int k0, int n, int step, F&& part) {
  const int lane = threadIdx.x & 31;
  Joined j = {-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  // eight parts' loads in flight
  constexpr int U = 8;
  for (int k = k0; k < n; k += U * step) {
    float2 v[U];
    float4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      v[i] = make_float2(-INFINITY, 0.f);
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k + i * step < n) {
        const float2* ml;
        const float* acc;
        part(k + i * step, ml, acc);
        v[i] = __ldcg(ml);
        x[i] = __ldcg(reinterpret_cast<const float4*>(acc) + lane);
      }
    }
    float M = j.M;
#pragma unroll
    for (int i = 0; i < U; ++i) M = fmaxf(M, v[i].x);
    const float ref = M == -INFINITY ? 0.f : M, a = ex2f_(j.M - ref);
    j.M = M;
    j.L *= a;
#pragma unroll
    for (int c = 0; c < 4; ++c) j.o[c] *= a;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float f = ex2f_(v[i].x - ref);
      j.L += v[i].y * f;
      j.o[0] += x[i].x * f;
      j.o[1] += x[i].y * f;
      j.o[2] += x[i].z * f;
      j.o[3] += x[i].w * f;
    }
  }
  return j;
}

// All eight warps of the CTA on one row.
template <class F>
__device__ __forceinline__ Joined join_parts_cta(JoinScratch* sc, int n, F&& part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Joined mine = join_parts(warp, n, kJoinWarps, part);
  __syncthreads();  // the row before has been read
  if (lane == 0) sc->ml[warp] = make_float2(mine.M, mine.L);
  *reinterpret_cast<float4*>(sc->o[warp] + 4 * lane) = make_float4(mine.o[0], mine.o[1], mine.o[2], mine.o[3]);
  __syncthreads();
  Joined j = {-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) j.M = fmaxf(j.M, sc->ml[w].x);
  const float ref = j.M == -INFINITY ? 0.f : j.M;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = ex2f_(sc->ml[w].x - ref);
    const float4 x = *reinterpret_cast<const float4*>(sc->o[w] + 4 * lane);
    j.L += sc->ml[w].y * f;
    j.o[0] += x.x * f;
    j.o[1] += x.y * f;
    j.o[2] += x.z * f;
    j.o[3] += x.w * f;
  }
  return j;
}

template <bool BF16>
__device__ __forceinline__ void write_row(uint16_t* out, const Joined& j) {
  const float inv = j.L > 0.f ? 1.f / j.L : j.L == 0.f ? 0.f : j.L;
  *reinterpret_cast<uint2*>(out + 4 * (threadIdx.x & 31)) =
      make_uint2(pack2<BF16>(j.o[0] * inv, j.o[1] * inv), pack2<BF16>(j.o[2] * inv, j.o[3] * inv));
}

// Without a prefix: CTA (x, y) joins the rows from y * STEP on (STEP 1 or 8 of
// them) of the unit that attention CTA x began and a later one ended.
// Everything else is in the output already.
template <bool BF16, int STEP>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_units_kernel(const AttnParams a) {
  __shared__ JoinScratch sc;
  const int warp = threadIdx.x >> 5, c = blockIdx.x;
  grid_dep_wait();
  const UnitMeta* u = a.part.begun + c;
  const int rows = __ldcg(&u->rows), r0 = blockIdx.y * STEP;
  if (r0 >= rows) return;
  const int n = __ldcg(&u->parts);
  UnitMeta m = {};
  m.tok = __ldcg(&u->tok);
  m.g0 = __ldcg(&u->g0);
  m.kh = __ldcg(&u->kh);
  const int R = a.part.R;
  int r = 0;
  auto part = [&](int k, const float2*& ml, const float*& acc) {
    const long long rec = (long long)(2 * (c + k) + (k == 0)) * R + r;
    ml = a.part.ml + rec;
    acc = a.part.acc + rec * kHeadDim;
  };
  auto out = [&] { return a.out + row_index(a, m, r) * kHeadDim; };
  if (STEP > 1 && n <= kJoinFew) {
    r = r0 + warp;
    if (r < rows) write_row<BF16>(out(), join_parts(0, n, 1, part));
  } else {
    for (r = r0; r < min(rows, r0 + STEP); ++r) {
      const Joined j = join_parts_cta(&sc, n, part);
      if (warp == 0) write_row<BF16>(out(), j);
    }
  }
}

// With a prefix: every row has a part or more of it, and of its own keys.
// Ticks of a sequence's own units before row tile `rts`, added up by a whole warp: a long chunk has hundreds of row
// tiles, and every row's join asks.
template <int R>
__device__ __forceinline__ long long seq_ticks_warp(const SeqSpan& s, int rts, int Gq, int S0, int kv_heads) {
  long long t = 0;
  for (int rt = threadIdx.x & 31; rt < rts; rt += 32) t += unit_ticks<R>(R, own_tiles(s, rt * R, R, Gq, S0));
  if (rts) {
#pragma unroll
    for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
  }
  return t * kv_heads;
}

template <int R>
__device__ __forceinline__ void own_place(const AttnParams& a, const SeqSpan& s, int b, int kh, int lr, long long* f,
                                          int* n, int* t) {
  const int rt = lr / R, rows = min(R, s.n * a.Gq - rt * R);
  *n = own_tiles(s, rt * R, rows, a.Gq, a.S0);
  *t = LineCost<R>::tile(rows);
  *f = __ldcg(a.part.plan + 1 + b) + seq_ticks_warp<R>(s, rt, a.Gq, a.S0, a.c.kv_heads) + kh * unit_ticks<R>(rows, *n) +
       LineCost<R>::unit(rows);
}
template <int R>
__device__ __forceinline__ void prefix_place(const AttnParams& a, int kh, int lr, long long* f, int* n, int* t) {
  const int all_rows = a.N * a.Gq, rts = (all_rows + R - 1) / R, rt = lr / R;
  *n = prefix_tiles_of((int)__ldcg(a.prefix.plan + 1 + a.c.batch));
  const int rows = min(R, all_rows - rt * R);
  *t = LineCost<R>::tile(rows);
  *f = kh * prefix_ticks<R>(all_rows, rts, *n) + prefix_ticks<R>(all_rows, rt, *n) + LineCost<R>::unit(rows);
}

template <bool BF16, int STEP>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_rows_kernel(const AttnParams a) {
  __shared__ JoinScratch sc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row_first = (long long)blockIdx.x * STEP, rows_all = (long long)a.N * a.Hq;
  // Where a row's parts lie: CTAs first .. first + n - 1 of the launch that had its unit, or one record of the row.
  struct Parts {
    int first, n, r;
  };
  struct Row {
    Parts pre, own;
    bool live;  // there is something to write
    long long row;
    int b, i, kh, gi;  // i < 0: it sees nothing
    SeqSpan s;
  };
  const int end = __ldg(a.offsets + a.c.batch);
  auto find = [&](long long row) {  // from the call's inputs alone
    Row w = {};
    w.row = row;
    w.i = -1;
    if (row >= rows_all) return w;
    const int tok = (int)(row / a.Hq), h = (int)(row - (long long)tok * a.Hq);
    if (tok >= end) return w;
    w.live = true;
    w.kh = h / a.Gq;
    w.gi = h - w.kh * a.Gq;
    w.b = find_sequence(a.offsets, a.c.batch, tok, lane & 15, (lane & 16) ? 0xffff0000u : 0x0000ffffu);
    unsigned bad = 0;
    w.s = seq_span(a, w.b, &bad);
    const int i = tok - w.s.tok0;
    if (i >= 0 && i < w.s.n && row_limit(w.s, i) > 0) w.i = i;
    return w;
  };
  auto place = [&](Row& w) {  // from the attention's plan
    if (w.i < 0) return;
    const SeqSpan& s = w.s;
    const int b = w.b, kh = w.kh, gi = w.gi, i = w.i, tok = s.tok0 + i;
    auto parts = [](const PartSet& ps, long long f, int n, int t, int r) {
      const long long W = __ldcg(ps.plan);
      const int first = div_small(f, W);
      return Parts{first, n ? div_small(f + (long long)(n - 1) * t, W) - first + 1 : 0, r};
    };
    long long f;
    int n, t;
    const int lr = i * a.Gq + gi, gr = tok * a.Gq + gi;
    if (a.part.R == 8) own_place<8>(a, s, b, kh, lr, &f, &n, &t);
    else if (a.part.R == 16) own_place<16>(a, s, b, kh, lr, &f, &n, &t);
    else own_place<kManyRows>(a, s, b, kh, lr, &f, &n, &t);
    w.own = parts(a.part, f, n, t, lr % a.part.R);
    if (a.prefix.R == 8) prefix_place<8>(a, kh, gr, &f, &n, &t);
    else if (a.prefix.R == 16) prefix_place<16>(a, kh, gr, &f, &n, &t);
    else prefix_place<kManyRows>(a, kh, gr, &f, &n, &t);
    w.pre = parts(a.prefix, f, n, t, gr % a.prefix.R);
  };
  Row w = find(row_first + (STEP > 1 ? warp : 0));
  grid_dep_wait();
  auto part = [&](int k, const float2*& ml, const float*& acc) {
    const bool pre = k < w.pre.n;
    const PartSet& ps = pre ? a.prefix : a.part;
    const Parts& q = pre ? w.pre : w.own;
    const int c = pre ? k : k - w.pre.n;
    const bool whole = q.n == 1;
    const long long rec = whole ? (pre ? 0 : rows_all) + w.row : (long long)(2 * (q.first + c) + (c == 0)) * ps.R + q.r;
    ml = (whole ? a.row_ml : ps.ml) + rec;
    acc = (whole ? a.row_acc : ps.acc) + rec * kHeadDim;
  };
  if (STEP > 1) {
    place(w);
    if (!__syncthreads_or(w.pre.n + w.own.n > kJoinFew)) {
      if (w.live) write_row<BF16>(a.out + w.row * kHeadDim, join_parts(0, w.pre.n + w.own.n, 1, part));
      return;
    }
  }
  for (int r = 0; r < STEP; ++r) {
    if (STEP > 1) w = find(row_first + r);
    place(w);
    const Joined j = join_parts_cta(&sc, w.pre.n + w.own.n, part);
    if (warp == 0 && w.live) write_row<BF16>(a.out + w.row * kHeadDim, j);
  }
}

// ------------------------------------------------------------------ host

using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static TensorMapEncode tensor_map_encode() {
  static TensorMapEncode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<TensorMapEncode>(f);
  }();
  return fn;
}

// The pool as [page][head][token][channel]; a copy takes one page of one head, 64 channels.
static palu_status page_map(CUtensorMap* map, const palu_paged_cache* c, const void* base, const int64_t* strides) {
  TensorMapEncode encode = tensor_map_encode();
  if (!encode) return fail(PALU_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)c->page_size, (cuuint64_t)c->kv_heads, (cuuint64_t)c->n_pages};
  const cuuint64_t str[3] = {(cuuint64_t)strides[2] * 2, (cuuint64_t)strides[1] * 2, (cuuint64_t)strides[0] * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)c->page_size, 1, 1}, one[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, c->dtype == PALU_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, const_cast<void*>(base), dims, str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PALU_ERR_CUDA, "cuTensorMapEncodeTiled refused the pages' strides (" + std::to_string(r) + ")");
  return PALU_OK;
}

// Sizes that the host can know: which kernel takes the shared and which the
// own keys, and the workspace's parts.
struct AttnLayout {
  bool shared;       // the prefix is a part of its own
  bool both;         // its rows are many and the own units' few: a line of each
  int R_prefix, R_own;
  size_t plan_p, begun_p, ml_p, acc_p, plan_o, begun_o, ml_o, acc_o, row_ml, row_acc, total;
};

// Whether reading the shared pages once pays.  It saves the tiles that the sequences would each read (a row tile each at
// least) beyond those of the whole batch's row tiles; it costs a longer beginning and, for every row, a record of each
// part that is written, read and joined.  28 heads of 4 KV heads, 512 own keys, bf16, read once and by each sequence: 16
// sequences of 1 token behind 1024 keys 16.5 and 14.5 us, behind 4096 20.1 and 23.9; 256 sequences of 5 behind 256 128 and
// 96 us, behind 4096 182 and 353; 16 of 1024 new tokens behind 8192 1972 and 1456.  In clocks, summed over the SMs:
constexpr double kShareTile = 2900., kShareRow = 350., kShareLaunch = 13300.;

// The most new tokens a call for which it can (the tiles saved are at most one a sequence, KV head and tile of the table).
static int64_t most_shared_tokens(const palu_paged_cache* c, int32_t q_heads) {
  const double tiles = prefix_tiles_of(c->table_width * c->page_size);
  const double n = (kShareTile * c->kv_heads * tiles * c->batch - kShareLaunch * device_sm_count()) / (kShareRow * q_heads);
  return std::max<int64_t>(1, (int64_t)n);
}
static bool share_pays(const palu_paged_cache* c, int64_t tokens, int32_t q_heads, int32_t max_new, int32_t shared_pages) {
  if (shared_pages == 0 || c->batch == 1 || tokens > most_shared_tokens(c, q_heads)) return false;
  const int Gq = q_heads / c->kv_heads;
  auto row_tiles = [&](double new_tokens) { return ceil(new_tokens * Gq / kManyRows); };
  // the counts are the device's: as many sequences as can be with the most new tokens, one token for the others
  const double many = std::min<int64_t>(max_new, tokens), B = std::min<int64_t>(c->batch, tokens);
  const double full = many > 1 ? std::min(B, (tokens - B) / (many - 1)) : 0;
  const double saved = full * row_tiles(many) + (B - full) * row_tiles(1) - row_tiles((double)tokens);
  return kShareTile * c->kv_heads * prefix_tiles_of(shared_pages * c->page_size) * saved >
         kShareRow * (double)tokens * q_heads + kShareLaunch * device_sm_count();
}

static palu_status attn_layout(const palu_paged_cache* c, int64_t tokens, int32_t q_heads, int32_t max_new,
                               int32_t shared_pages, AttnLayout* l) {
  palu_status st = paged_check(c);
  if (st != PALU_OK) return st;
  if (tokens < 1 || q_heads < 1 || max_new < 1) return fail(PALU_ERR_INVALID_ARG, "tokens, q_heads and max_new must be positive");
  if (q_heads % c->kv_heads) return fail(PALU_ERR_INVALID_ARG, "q_heads must be a multiple of the cache's kv_heads");
  const int Gq = q_heads / c->kv_heads;
  if (Gq > kMaxPagedGq) return fail(PALU_ERR_UNSUPPORTED, "at most 64 query heads per KV head");
  if (tokens > (1LL << 31) / q_heads - 256) return fail(PALU_ERR_UNSUPPORTED, "too many tokens for one call");
  if (shared_pages < 0 || shared_pages > c->table_width)
    return fail(PALU_ERR_INVALID_ARG, "shared_pages must be in [0, table_width]");
  const int64_t own_rows = std::min<int64_t>(max_new, tokens) * Gq, all_rows = tokens * Gq;
  l->shared = share_pays(c, tokens, q_heads, max_new, shared_pages);
  l->R_prefix = all_rows <= 8 ? 8 : all_rows <= 16 ? 16 : kManyRows;
  const int R_rows = own_rows <= 8 ? 8 : own_rows <= 16 ? 16 : kManyRows;
  // Otherwise one line: up to 16 rows in all go to the prefix's row tiles, and so do own units of more than 16.
  l->both = l->shared && l->R_prefix == kManyRows && R_rows < kManyRows && device_sm_count() > 1;
  l->R_own = l->shared && !l->both ? l->R_prefix : R_rows;
  const size_t slots = 2 * (size_t)device_sm_count();
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  auto take_parts = [&](int R, size_t* plan, size_t* begun, size_t* ml, size_t* acc) {
    *plan = take(sizeof(long long) * (2 + (size_t)c->batch));
    *begun = take(slots / 2 * sizeof(UnitMeta));
    *ml = take(slots * R * sizeof(float2));
    *acc = take(slots * R * kHeadDim * sizeof(float));
  };
  // With shared pages the size is the same whether or not they are read once here: it also serves fewer tokens, and
  // any other number of them.
  const bool may_share = shared_pages > 0 && c->batch > 1;
  const size_t records = may_share ? 2 * (size_t)std::min(tokens, most_shared_tokens(c, q_heads)) * q_heads : 0;
  l->row_ml = take(records * sizeof(float2));
  l->row_acc = take(records * kHeadDim * sizeof(float));
  const size_t parts = o;
  take_parts(l->R_own, &l->plan_o, &l->begun_o, &l->ml_o, &l->acc_o);
  if (l->both) take_parts(l->R_prefix, &l->plan_p, &l->begun_p, &l->ml_p, &l->acc_p);
  l->total = o;
  if (may_share) {
    size_t unused;
    o = parts;
    take_parts(R_rows, &unused, &unused, &unused, &unused);
    take_parts(l->R_prefix, &unused, &unused, &unused, &unused);
    l->total = o;
  }
  return PALU_OK;
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_paged_attn_workspace_size(const palu_paged_cache* cache, int64_t tokens, int32_t q_heads,
                                                      int32_t max_new, int32_t shared_pages, size_t* bytes) {
  AttnLayout l;
  palu_status st = attn_layout(cache, tokens, q_heads, max_new, shared_pages, &l);
  if (st != PALU_OK) return st;
  if (!bytes) return fail(PALU_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = l.total;
  return PALU_OK;
}

extern "C" palu_status palu_paged_attn(const palu_paged_cache* cache, int64_t tokens, const int32_t* offsets,
                                       int32_t max_new, int32_t q_heads, const void* q, const int64_t q_strides[2],
                                       int32_t shared_pages, float softmax_scale, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  AttnLayout l;
  palu_status st = attn_layout(cache, tokens, q_heads, max_new, shared_pages, &l);
  if (st != PALU_OK) return st;
  if (!q || !q_strides || !offsets || !out || !workspace) return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15 || (uintptr_t)offsets & 3)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be 16-byte aligned (offsets 4)");
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] < 0 || q_strides[i] % 8)
      return fail(PALU_ERR_INVALID_ARG, "q's strides must be non-negative multiples of 8 elements");
  const int64_t qe[2] = {tokens, q_heads};
  if (rows_overlap(out, tokens * q_heads, q, q_strides, qe, 2)) return fail(PALU_ERR_INVALID_ARG, "out overlaps q");
  if (!(softmax_scale >= 0.f) || isinf(softmax_scale))
    return fail(PALU_ERR_INVALID_ARG, "softmax_scale must be finite and not negative");
  if (workspace_bytes < l.total) return fail(PALU_ERR_INVALID_ARG, "workspace too small");
  CUtensorMap km, vm;
  if ((st = page_map(&km, cache, cache->k_pages, cache->k_strides)) != PALU_OK ||
      (st = page_map(&vm, cache, cache->v_pages, cache->v_strides)) != PALU_OK)
    return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnParams p = {};
  p.c = paged_view(cache);
  p.q = static_cast<const uint16_t*>(q);
  p.qs0 = q_strides[0], p.qs1 = q_strides[1];
  p.offsets = offsets;
  p.out = static_cast<uint16_t*>(out);
  p.row_ml = reinterpret_cast<float2*>(ws + l.row_ml);
  p.row_acc = reinterpret_cast<float*>(ws + l.row_acc);
  p.N = (int)tokens;
  p.max_new = max_new;
  p.Hq = q_heads;
  p.Gq = q_heads / cache->kv_heads;
  p.gq_mul = (65536 + p.Gq - 1) / p.Gq;
  p.S0 = l.shared ? shared_pages * cache->page_size : 0;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)kHeadDim)) * 1.4426950408889634f;
  p.part = {reinterpret_cast<float2*>(ws + l.ml_o), reinterpret_cast<float*>(ws + l.acc_o),
            reinterpret_cast<long long*>(ws + l.plan_o), reinterpret_cast<UnitMeta*>(ws + l.begun_o), l.R_own};
  p.prefix = p.part;
  if (l.both)
    p.prefix = {reinterpret_cast<float2*>(ws + l.ml_p), reinterpret_cast<float*>(ws + l.acc_p),
                reinterpret_cast<long long*>(ws + l.plan_p), reinterpret_cast<UnitMeta*>(ws + l.begun_p), l.R_prefix};
  const bool bf16 = cache->dtype == PALU_TYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto* const attend = l.both ? launch_both : l.R_own == kManyRows ? launch_many : launch_few;
  if ((st = attend(p, km, vm, bf16, s)) != PALU_OK) return st;
  if (!l.shared) {
    if (l.R_own < kManyRows) {
      const dim3 jgrid(device_sm_count(), l.R_own);
      return bf16 ? launch(paged_join_units_kernel<true, 1>, jgrid, 32 * kJoinWarps, 0, true, s, "paged_join_units_kernel launch", p)
                  : launch(paged_join_units_kernel<false, 1>, jgrid, 32 * kJoinWarps, 0, true, s, "paged_join_units_kernel launch", p);
    }
    const dim3 jgrid(device_sm_count(), l.R_own / kJoinWarps);
    return bf16 ? launch(paged_join_units_kernel<true, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                         "paged_join_units_kernel launch", p)
                : launch(paged_join_units_kernel<false, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                         "paged_join_units_kernel launch", p);
  }
  const long long rows = (long long)p.N * p.Hq;
  if (rows <= kJoinRows)
    return bf16 ? launch(paged_join_rows_kernel<true, 1>, dim3((unsigned)rows), 32 * kJoinWarps, 0, true, s,
                         "paged_join_rows_kernel launch", p)
                : launch(paged_join_rows_kernel<false, 1>, dim3((unsigned)rows), 32 * kJoinWarps, 0, true, s,
                         "paged_join_rows_kernel launch", p);
  const dim3 jgrid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
  return bf16 ? launch(paged_join_rows_kernel<true, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                       "paged_join_rows_kernel launch", p)
              : launch(paged_join_rows_kernel<false, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                       "paged_join_rows_kernel launch", p);
}
