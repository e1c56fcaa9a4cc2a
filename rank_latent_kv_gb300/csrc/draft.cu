// Verification of drafted tokens from given random numbers.
//
// One cluster of 8 CTAs per sequence.  Every CTA repeats the (few) acceptance
// tests, so all know the number kept, a; then the cluster reads the one row
// of the target and the one of the draft that the drawn token depends on,
// each once: V * 8 bytes a sequence are all that the call has to move.
//
// The token is the first whose running sum of w(t) = max(p(t) - q(t), 0)
// passes u * total.  With 150,000 tokens most gaps between running sums are
// far below one fp32 ulp of the total, so fp32 sums would pick other tokens
// than the exact sums; fp64 sums would be right, but cost five fp64
// instructions a value at 2 lanes a clock and SM: about 80 us for 64
// rows of 152,065, against 12 us of reading.  So each lane keeps an unevaluated
// pair of floats: the difference as its rounded value and exact remainder,
// the sum with its error terms (about 17 fp32 instructions a value); fp64
// starts with one value per lane.  The pair is right to about 2^-46 of the sum.
#include <algorithm>

#include "draft.h"
#include "palu_internal.cuh"

namespace palu {

constexpr int kDraftCluster = 8;
constexpr int kDraftWarps = 16;
constexpr int kDraftThreads = 32 * kDraftWarps;
constexpr int kDraftSegs = kDraftCluster * kDraftWarps;  // a row is cut into one segment a warp
constexpr int kDraftMax = 256;

struct DraftParams {
  const float *target, *draft;
  long long ts0, ts1, ds0, ds1;
  const long long* drafts;
  const int* n_drafts;
  const float *accept_u, *sample_u;
  const long long* lengths;
  long long* tokens;
  int* n_kept;
  long long* new_lengths;
  int k, V;
  int seg;  // values a segment
};

// The weight of a value as an unevaluated pair (hi + lo exactly p - q), or
// (0, 0) where it is not positive or not a number.
__device__ __forceinline__ void draft_weight(float p, float q, float& hi, float& lo) {
  two_sum(p, -q, hi, lo);
  if (!(hi > 0.f)) hi = lo = 0.f;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote_f64(double* local, uint32_t rank, double v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

__global__ void __cluster_dims__(kDraftCluster, 1, 1) __launch_bounds__(kDraftThreads, 2)
    draft_verify_kernel(const DraftParams d) {
  __shared__ double sums[2][kDraftSegs];  // one set a pass: the second pass never waits for readers of the first
  __shared__ double wsum[kDraftWarps];
  __shared__ int first_out;   // first draft that is not kept
  __shared__ int found;       // drawn token
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const long long b = blockIdx.x / kDraftCluster;
  const int n = d.n_drafts ? min(max(d.n_drafts[b], 0), d.k) : d.k;
  if (tid == 0) {
    first_out = n;
    found = 0x7fffffff;
  }
  __syncthreads();
  if (tid < n) {
    const long long x = d.drafts[b * d.k + tid];
    bool keep = false;
    if (x >= 0 && x < d.V) {
      const float p = d.target[b * d.ts0 + tid * d.ts1 + x];
      const float q = d.draft ? d.draft[b * d.ds0 + tid * d.ds1 + x] : 1.f;
      // 24 x 24 bits: the product is exact in fp64
      keep = (double)d.accept_u[b * d.k + tid] * (double)q < (double)p;
    }
    if (!keep) atomicMin(&first_out, tid);
  }
  __syncthreads();
  const int a = first_out;
  const float* prow = d.target + b * d.ts0 + a * d.ts1;
  const float* qrow = (a < n && d.draft) ? d.draft + b * d.ds0 + a * d.ds1 : nullptr;
  // without draft probabilities the refused token itself has weight 0
  long long skip = (a < n && !d.draft) ? d.drafts[b * d.k + a] : -1;
  const int seg0 = (int)rank * kDraftWarps + warp;
  const long long t0 = (long long)seg0 * d.seg, t1 = min(t0 + d.seg, (long long)d.V);
  double total = 0.0, before = 0.0;
  int win = -1;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float s = 0.f, e = 0.f;
    long long t = t0 + lane;
    // eight loads of each row in flight a lane
    for (; t + 7 * 32 < t1; t += 8 * 32) {
      float p[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = prow[t + 32 * i];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = qrow ? qrow[t + 32 * i] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float hi, lo, r;
        draft_weight(t + 32 * i == skip ? 0.f : p[i], q[i], hi, lo);
        two_sum(s, hi, s, r);
        e = __fadd_rn(e, __fadd_rn(r, lo));
      }
    }
    for (; t < t1; t += 32) {
      float hi, lo, r;
      draft_weight(t == skip ? 0.f : prow[t], qrow ? qrow[t] : 0.f, hi, lo);
      two_sum(s, hi, s, r);
      e = __fadd_rn(e, __fadd_rn(r, lo));
    }
    double sum = (double)s + (double)e;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane < kDraftCluster) store_remote_f64(&sums[pass][seg0], lane, sum);
    cluster_sync();
    // every warp finds the segment of the drawn token: four segments a lane
    double v[kDraftSegs / 32], run = 0.0;
#pragma unroll
    for (int i = 0; i < kDraftSegs / 32; ++i) run += (v[i] = sums[pass][lane * (kDraftSegs / 32) + i]);
    double incl = run;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const double target = (double)d.sample_u[b] * total;
    double c = incl - run;
    int mine = kDraftSegs;
    double mine_before = 0.0;
#pragma unroll
    for (int i = 0; i < kDraftSegs / 32; ++i) {
      if (mine == kDraftSegs && v[i] > 0.0 && c + v[i] > target) {
        mine = lane * (kDraftSegs / 32) + i;
        mine_before = c;
      }
      c += v[i];
    }
    const unsigned hit = __ballot_sync(0xffffffffu, mine < kDraftSegs);
    if (hit) {
      const int src = __ffs(hit) - 1;
      win = __shfl_sync(0xffffffffu, mine, src);
      before = __shfl_sync(0xffffffffu, mine_before, src);
      break;
    }
    // no weight over zero: the target's own row, once (the refused token counts again)
    if (a == n) break;
    qrow = nullptr;
    skip = -1;
  }
  // the CTA that holds the segment (or the first one, without any) answers
  if (win >= 0 ? (win / kDraftWarps != (int)rank) : (rank != 0)) return;
  int token = -1;
  if (win >= 0) {
    const double target = (double)d.sample_u[b] * total;
    const long long w0 = (long long)win * d.seg, w1 = min(w0 + d.seg, (long long)d.V);
    const int per = (int)((w1 - w0 + kDraftThreads - 1) / kDraftThreads);
    // `per` consecutive values a thread, their sums scanned over the CTA
    const long long a0 = w0 + (long long)tid * per, a1 = min(a0 + per, w1);
    double own = 0.0;
    int last = -1;
    for (long long t = a0; t < a1; ++t) {
      float hi, lo;
      draft_weight(t == skip ? 0.f : prow[t], qrow ? qrow[t] : 0.f, hi, lo);
      if (hi > 0.f) last = (int)t;
      own += (double)hi + (double)lo;
    }
    double incl = own;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    double c = before + (incl - own);
    for (int w = 0; w < warp; ++w) c += wsum[w];
    for (long long t = a0; t < a1; ++t) {
      float hi, lo;
      draft_weight(t == skip ? 0.f : prow[t], qrow ? qrow[t] : 0.f, hi, lo);
      c += (double)hi + (double)lo;
      if (hi > 0.f && c > target) {
        atomicMin(&found, (int)t);
        break;
      }
    }
    __syncthreads();
    token = found;
    // the segment's sum passed the target, its rescan by another order of summation may stop one rounding short of it:
    // then it is the segment's last value with a weight
    if (token == 0x7fffffff) {
      __syncthreads();
      if (tid == 0) found = -1;
      __syncthreads();
      if (last >= 0) atomicMax(&found, last);
      __syncthreads();
      token = found;
    }
  }
  for (int i = tid; i <= d.k; i += kDraftThreads)
    d.tokens[b * (d.k + 1) + i] = i < a ? d.drafts[b * d.k + i] : i == a ? token : -1;
  if (tid == 0) {
    d.n_kept[b] = a;
    if (d.lengths) d.new_lengths[b] = d.lengths[b] - (n - a);
  }
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_draft_verify(int64_t batch, int32_t k, int64_t vocab, const float* target,
                                         const int64_t target_strides[2], const float* draft,
                                         const int64_t draft_strides[2], const int64_t* drafts,
                                         const int32_t* n_drafts, const float* accept_u, const float* sample_u,
                                         const int64_t* lengths, int64_t* tokens, int32_t* n_kept,
                                         int64_t* new_lengths, void* stream) {
  if (batch < 1 || batch > (1 << 24)) return fail(PALU_ERR_INVALID_ARG, "batch must be in [1, 2^24]");
  if (k < 1 || k > kDraftMax) return fail(PALU_ERR_UNSUPPORTED, "k must be in [1, 256]");
  if (vocab < 1 || vocab > 0x7ffffffe) return fail(PALU_ERR_INVALID_ARG, "vocab must be in [1, 2^31 - 2]");
  if (!target || !target_strides || !drafts || !accept_u || !sample_u || !tokens || !n_kept)
    return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if (draft && !draft_strides) return fail(PALU_ERR_INVALID_ARG, "draft_strides is NULL");
  if (!lengths != !new_lengths) return fail(PALU_ERR_INVALID_ARG, "lengths and new_lengths come together");
  if (tokens == drafts) return fail(PALU_ERR_INVALID_ARG, "tokens must not be the drafts' array");
  if (target_strides[0] < 0 || target_strides[1] < 0 || (draft && (draft_strides[0] < 0 || draft_strides[1] < 0)))
    return fail(PALU_ERR_INVALID_ARG, "strides must not be negative");
  if (((uintptr_t)target | (uintptr_t)draft | (uintptr_t)accept_u | (uintptr_t)sample_u | (uintptr_t)n_kept |
       (uintptr_t)n_drafts) & 3 ||
      ((uintptr_t)drafts | (uintptr_t)tokens | (uintptr_t)lengths | (uintptr_t)new_lengths) & 7)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  DraftParams p;
  p.target = target;
  p.draft = draft;
  p.ts0 = target_strides[0];
  p.ts1 = target_strides[1];
  p.ds0 = draft ? draft_strides[0] : 0;
  p.ds1 = draft ? draft_strides[1] : 0;
  p.drafts = reinterpret_cast<const long long*>(drafts);
  p.n_drafts = n_drafts;
  p.accept_u = accept_u;
  p.sample_u = sample_u;
  p.lengths = reinterpret_cast<const long long*>(lengths);
  p.tokens = reinterpret_cast<long long*>(tokens);
  p.n_kept = n_kept;
  p.new_lengths = reinterpret_cast<long long*>(new_lengths);
  p.k = k;
  p.V = (int)vocab;
  p.seg = (int)((vocab + kDraftSegs - 1) / kDraftSegs);
  draft_verify_kernel<<<(unsigned)(batch * kDraftCluster), kDraftThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cuda_check(cudaGetLastError(), "draft_verify_kernel launch");
}
