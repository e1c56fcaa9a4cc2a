// Pages handed out and taken back on the device (include/pages.h).
//
// Whole numbers and a few kilobytes: bound by latency, so everything is one
// launch of one CTA, or, where there are many rows to write, of a cluster.
// Every CTA reads all counts and lengths and finds all sums itself (a scan in
// shared memory); the cluster meets, and only then is anything written.  What
// is written is flat: the k-th page given back, the k-th page taken, the k-th
// new row, so that one sequence with thousands of pages is as even as thousands
// of sequences with one.  Each finds its sequence by a search in the sums; a
// lane's four lookups are under way together.  (One search for a warp's 128
// entries and a walk from there is a fifth faster for 512 sequences with 66,000
// rows, half as fast for 4,096 with 35,000, and its code costs the smallest calls
// 2 us; the host takes longer than either.)
// Pages given back may be taken by the same call, so the cluster meets between
// the two, and once more before the rows look pages up.  16 sequences take 5 us a
// plan, 512 with 66,000 rows 20.
#include <cooperative_groups.h>

#include "pages.h"
#include "palu_internal.cuh"

namespace palu {

constexpr int32_t kPoolMagic = 0x504F4F4C;  // "POOL"
constexpr int kPlanThreads = 512;
constexpr int kPlanCtas = 8;                // of a cluster
constexpr int kPlanBatch = 4096;
constexpr long long kPlanAlone = 4096;      // rows up to which one CTA is as fast
constexpr int kPlanRun = 4;                 // rows, or pages, that a thread takes at once
// offsets, pages given and taken before each sequence; pages needed and held, lengths before the call
constexpr int plan_smem(int64_t batch) { return (int)(3 * (batch + 1) + 3 * batch) * 4; }

struct PlanParams {
  int* table;
  long long* lengths;
  int *held, *free_pages, *n_free;
  unsigned* error;
  const int* counts;
  int* offsets;
  long long *positions, *slots;
  long long n_pages, tokens;
  int batch, width, shared;
  unsigned page;
};

// The sequence with sums[b] <= k < sums[b + 1].
__device__ __forceinline__ int owner(const int* sums, int batch, int k) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ int smem[];
  __shared__ long long warp_sum[3][kPlanThreads / 32];
  __shared__ unsigned bad_s;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.batch;
  int *off = smem, *given = off + B + 1, *taken = given + B + 1, *need_s = taken + B + 1, *held_s = need_s + B, *len_s = held_s + B;
  if (tid == 0) bad_s = 0;
  __syncthreads();
  // each thread's sequences, and their sums
  const int per = (B + kPlanThreads - 1) / kPlanThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  unsigned bad = 0;
  long long sum[3] = {0, 0, 0};
  const int n_free = *p.n_free;
  if (n_free < 0 || n_free > p.n_pages) bad |= PALU_DEVERR_SPAN;
  for (int b = b0; b < b1; ++b) {
    const long long len = p.lengths[b];
    const int count = __ldg(p.counts + b), held = p.held[b];
    int need = held;
    if (count < 0 || len < 0 || held < 0 || held > p.width)
      bad |= PALU_DEVERR_SPAN;
    else if (len > (long long)p.width * (int)p.page - count)
      bad |= PALU_DEVERR_CAPACITY;
    else
      need = max((int)(((unsigned)(len + count) + p.page - 1) / p.page), min(held, p.shared));
    need_s[b] = need;
    held_s[b] = held;
    len_s[b] = (int)len;  // below 2^30 where the call is not refused
    sum[0] += max(count, 0);
    sum[1] += max(held - need, 0);
    sum[2] += max(need - held, 0);
  }
  long long before[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long x = sum[i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[i][warp] = x;
    before[i] = x - sum[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    total[i] = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) before[i] += warp_sum[i][w];
      total[i] += warp_sum[i][w];
    }
  }
  if (total[0] > p.tokens || n_free + total[1] > p.n_pages) bad |= PALU_DEVERR_SPAN;
  if (total[2] > n_free + total[1]) bad |= PALU_DEVERR_CAPACITY;
  if (bad) atomicOr(&bad_s, bad);
  __syncthreads();
  bad = bad_s;  // the same in every CTA of the cluster
  const long long first = (long long)cta * kPlanThreads + tid, step = (long long)ctas * kPlanThreads;
  if (bad) {
    if (cta == 0 && tid == 0) atomicOr(p.error, bad);
    for (long long i = first; i <= B; i += step) p.offsets[i] = 0;
    for (long long i = first; i < p.tokens; i += step) {
      if (p.positions) p.positions[i] = -1;
      if (p.slots) p.slots[i] = -1;
    }
    return;
  }
  // none of the sums is above 2^31 - 1: tokens and n_pages are not, and what is taken is at most what is free
  for (int b = b0; b < b1; ++b) {
    off[b] = (int)before[0];
    given[b] = (int)before[1];
    taken[b] = (int)before[2];
    before[0] += __ldg(p.counts + b);
    before[1] += max(held_s[b] - need_s[b], 0);
    before[2] += max(need_s[b] - held_s[b], 0);
  }
  if (tid == 0) {
    off[B] = (int)total[0];
    given[B] = (int)total[1];
    taken[B] = (int)total[2];
  }
  cluster.sync();  // all have read what is written from here on (and a CTA its sums)
  // What entry k < n reads, load(b, k - sums[b], k), and then what it writes, store(b, k - sums[b], k, value).
  auto each = [&](const int* sums, int n, auto&& load, auto&& store) {
    const int warps = (int)(step >> 5);
    for (long long k0 = (first >> 5) * (32 * kPlanRun); k0 < n; k0 += (long long)warps * (32 * kPlanRun)) {
      int bs[kPlanRun], value[kPlanRun];
#pragma unroll
      for (int i = 0; i < kPlanRun; ++i) {
        const int k = (int)min(k0 + 32 * i + lane, (long long)n - 1);
        bs[i] = owner(sums, B, k);
        value[i] = load(bs[i], k - sums[bs[i]], k);
      }
#pragma unroll
      for (int i = 0; i < kPlanRun; ++i) {
        const long long k = k0 + 32 * i + lane;
        if (k < n) store(bs[i], (int)k - sums[bs[i]], (int)k, value[i]);
      }
    }
  };
  // of a place (below 2^30): the page-table entry
  const int shift = p.page & (p.page - 1) ? -1 : 31 - __clz(p.page);
  auto entry_of = [&](unsigned place) { return shift >= 0 ? place >> shift : place / p.page; };
  each(
      given, (int)total[1], [&](int b, int i, int k) { return p.table[(long long)b * p.width + need_s[b] + i]; },
      [&](int b, int i, int k, int page) { p.free_pages[n_free + k] = page; });
  if (total[1]) cluster.sync();
  const long long top = n_free + total[1];
  each(
      taken, (int)total[2], [&](int b, int i, int k) { return __ldcg(p.free_pages + (top - 1 - k)); },
      [&](int b, int i, int k, int page) { p.table[(long long)b * p.width + held_s[b] + i] = page; });
  for (long long b = first; b < B; b += step) {
    p.held[b] = need_s[b];
    p.lengths[b] = len_s[b] + (off[b + 1] - off[b]);
  }
  for (long long i = first; i <= B; i += step) p.offsets[i] = off[i];
  if (cta == 0 && tid == 0) *p.n_free = (int)(top - total[2]);
  if (total[2]) cluster.sync();
  each(
      off, (int)total[0],
      [&](int b, int i, int k) { return p.slots ? __ldcg(p.table + (long long)b * p.width + entry_of(len_s[b] + i)) : 0; },
      [&](int b, int i, int k, int page) {
        const unsigned place = len_s[b] + i;
        if (p.positions) p.positions[k] = place;
        if (p.slots) p.slots[k] = (long long)page * p.page + (place - entry_of(place) * p.page);
      });
  for (long long k = total[0] + first; k < p.tokens; k += step) {
    if (p.positions) p.positions[k] = -1;
    if (p.slots) p.slots[k] = -1;
  }
}

static palu_status pool_check(const palu_page_pool* pool) {
  if (!pool) return fail(PALU_ERR_INVALID_ARG, "pool is NULL");
  if (pool->magic != kPoolMagic) return fail(PALU_ERR_NOT_INITIALIZED, "page pool is not initialised");
  return PALU_OK;
}

// Whether two byte ranges share memory.
static bool ranges_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_page_pool_init(palu_page_pool* pool, int32_t page_size, int64_t batch, int64_t table_width,
                                           int64_t n_pages, int32_t* page_table, int64_t* lengths, int32_t* held,
                                           int32_t* free_pages, int32_t* n_free, uint32_t* error) {
  if (!pool) return fail(PALU_ERR_INVALID_ARG, "pool is NULL");
  pool->magic = 0;
  if (page_size < 1 || page_size > 65536) return fail(PALU_ERR_UNSUPPORTED, "page_size must be in [1, 65536]");
  if (batch < 1 || table_width < 1) return fail(PALU_ERR_INVALID_ARG, "batch and table_width must be positive");
  if (batch > kPlanBatch) return fail(PALU_ERR_UNSUPPORTED, "at most 4096 sequences");
  if (table_width > (1LL << 30) / page_size) return fail(PALU_ERR_UNSUPPORTED, "at most 2^30 tokens a sequence");
  if (n_pages < 0 || n_pages > 0x7fffffff) return fail(PALU_ERR_INVALID_ARG, "n_pages must be in [0, 2^31)");
  if (!page_table || !lengths || !held || !n_free || !error || (!free_pages && n_pages))
    return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if (((uintptr_t)page_table | (uintptr_t)held | (uintptr_t)free_pages | (uintptr_t)n_free | (uintptr_t)error) & 3 ||
      (uintptr_t)lengths & 7)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  const void* arrays[6] = {page_table, lengths, held, free_pages, n_free, error};
  const int64_t bytes[6] = {batch * table_width * 4, batch * 8, batch * 4, n_pages * 4, 4, 4};
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (ranges_meet(arrays[i], bytes[i], arrays[j], bytes[j]))
        return fail(PALU_ERR_INVALID_ARG, "the pool's arrays must be disjoint");
  pool->page_size = page_size;
  pool->batch = (int32_t)batch;
  pool->table_width = (int32_t)table_width;
  pool->n_pages = n_pages;
  pool->page_table = page_table;
  pool->lengths = lengths;
  pool->held = held;
  pool->free_pages = free_pages;
  pool->n_free = n_free;
  pool->error = error;
  pool->magic = kPoolMagic;
  return PALU_OK;
}

extern "C" palu_status palu_page_plan(const palu_page_pool* pool, const int32_t* new_tokens, int64_t tokens,
                                      int32_t shared_pages, int32_t* offsets, int64_t* positions, int64_t* slots,
                                      void* stream) {
  palu_status st = pool_check(pool);
  if (st != PALU_OK) return st;
  if (tokens < 0 || tokens > 0x7fffffff) return fail(PALU_ERR_INVALID_ARG, "tokens must be in [0, 2^31)");
  if (shared_pages < 0 || shared_pages > pool->table_width)
    return fail(PALU_ERR_INVALID_ARG, "shared_pages must be in [0, table_width]");
  if (!new_tokens || !offsets) return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if (((uintptr_t)new_tokens | (uintptr_t)offsets) & 3 || ((uintptr_t)positions | (uintptr_t)slots) & 7)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  const int64_t B = pool->batch;
  const void* in[8] = {new_tokens,    pool->page_table, pool->lengths, pool->held,
                       pool->free_pages, pool->n_free,     pool->error,   nullptr};
  const int64_t in_bytes[8] = {B * 4, B * pool->table_width * 4, B * 8, B * 4, pool->n_pages * 4, 4, 4, 0};
  const void* out[3] = {offsets, positions, slots};
  const int64_t out_bytes[3] = {(B + 1) * 4, tokens * 8, tokens * 8};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 7; ++j)
      if (ranges_meet(out[i], out_bytes[i], in[j], in_bytes[j]))
        return fail(PALU_ERR_INVALID_ARG, "an output overlaps an input or the pool");
    for (int j = 0; j < i; ++j)
      if (ranges_meet(out[i], out_bytes[i], out[j], out_bytes[j])) return fail(PALU_ERR_INVALID_ARG, "the outputs overlap");
  }
  for (int j = 1; j < 7; ++j)
    if (ranges_meet(new_tokens, B * 4, in[j], in_bytes[j])) return fail(PALU_ERR_INVALID_ARG, "new_tokens overlaps the pool");
  PlanParams p = {};
  p.table = pool->page_table;
  p.lengths = reinterpret_cast<long long*>(pool->lengths);
  p.held = pool->held;
  p.free_pages = pool->free_pages;
  p.n_free = pool->n_free;
  p.error = pool->error;
  p.counts = new_tokens;
  p.offsets = offsets;
  p.positions = reinterpret_cast<long long*>(positions);
  p.slots = reinterpret_cast<long long*>(slots);
  p.n_pages = pool->n_pages;
  p.tokens = tokens;
  p.batch = pool->batch;
  p.width = pool->table_width;
  p.page = pool->page_size;
  p.shared = shared_pages;
  int per_sm = 0;
  if ((st = kernel_occupancy(reinterpret_cast<const void*>(page_plan_kernel), kPlanThreads, plan_smem(kPlanBatch), &per_sm)) != PALU_OK)
    return st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = tokens > kPlanAlone ? kPlanCtas : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attr.val.clusterDim.x);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem(B);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, page_plan_kernel, p), "page_plan_kernel launch");
}

extern "C" palu_status palu_page_pool_sync(const palu_page_pool* pool, uint32_t* device_error, void* stream) {
  palu_status st = pool_check(pool);
  if (st != PALU_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t e = 0;
  st = cuda_check(cudaMemcpyAsync(&e, pool->error, sizeof(e), cudaMemcpyDeviceToHost, s), "cudaMemcpyAsync(error word)");
  if (st != PALU_OK || (st = cuda_check(cudaStreamSynchronize(s), "cudaStreamSynchronize")) != PALU_OK) return st;
  if (device_error) *device_error = e;
  if (!e) return PALU_OK;
  if ((st = cuda_check(cudaMemsetAsync(pool->error, 0, sizeof(e), s), "cudaMemsetAsync(error word)")) != PALU_OK) return st;
  std::string msg = "device error word " + std::to_string(e) + ":";
  if (e & PALU_DEVERR_CAPACITY) msg += " too few free pages, or a length past the page table;";
  if (e & PALU_DEVERR_SPAN) msg += " a negative count or length, more new tokens than rows, or a count outside its array;";
  return fail(PALU_ERR_DEVICE, msg);
}
