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
// than the exact sums.  fp64 is no way out here: at 2 lanes a clock and SM the
// five fp64 instructions a value would take about 80 us for 64 rows of 152,065,
// against 12 us of reading.  So everything is an unevaluated pair of floats:
// a difference is its rounded value and the exact remainder, a sum carries its
// rounding errors along (about 18 fp32 instructions a value).
//
// How far a sum may be off, with u = 2^-24.  Eight values: seven remainders of
// at most u times the sum each are added up in one float, 49 u^2 at worst.  Two
// pairs: 3 u^2 of the result (16 u^2 of the eight values, whose remainder is not
// yet small).  A lane adds up nb groups of eight, then lanes, segments and CTAs
// follow in at most 18 sums of pairs: (66 + 3 nb + 54) u^2 with nb = V / 16384 at
// most.  The running sum of the drawn token adds the rescan of its segment, 36 +
// 6 nb, and what it is compared with is the total scaled, 2 more: together
// (278 + 12 nb) 2^-48 of the total, 2^-39 for 152,065 tokens.  (One remainder
// carried through a lane's whole stretch grew with its length instead: 2^-45 at
// 75 values a lane, but 2^-28 at 20,000.)
#include <algorithm>

#include "draft.h"
#include "palu_internal.cuh"

namespace palu {

constexpr int kDraftCluster = 8;
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
// Arrivals without an order of memory: enough to know that every CTA of the cluster has begun.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(float2* local, uint32_t rank, float2 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// Sums as pairs (x + y, |y| at most half an ulp of x).
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  float s, e, h, r;
  two_sum(a.x, b.x, s, e);
  e = __fadd_rn(e, __fadd_rn(a.y, b.y));
  two_sum(s, e, h, r);
  return make_float2(h, r);
}
__device__ __forceinline__ float2 pair_scale(float2 a, float u) {
  float p, e, h, r;
  two_prod(a.x, u, p, e);
  e = __fmaf_rn(a.y, u, e);
  two_sum(p, e, h, r);
  return make_float2(h, r);
}
__device__ __forceinline__ bool pair_above(float2 a, float2 b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }
__device__ __forceinline__ float2 shfl_up(float2 v, int x) {
  return make_float2(__shfl_up_sync(0xffffffffu, v.x, x), __shfl_up_sync(0xffffffffu, v.y, x));
}
__device__ __forceinline__ float2 shfl(float2 v, int src) {
  return make_float2(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src));
}
// Inclusive sums over the lanes.
__device__ __forceinline__ float2 warp_scan(float2 v, int lane) {
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const float2 y = shfl_up(v, x);
    if (lane >= x) v = pair_add(y, v);
  }
  return v;
}
// The sum before this lane.
__device__ __forceinline__ float2 before_lane(float2 incl, int lane) {
  const float2 y = shfl_up(incl, 1);
  return lane ? y : make_float2(0.f, 0.f);
}

// WARPS a CTA: a row is cut into one segment a warp of the cluster.
template <int WARPS>
__global__ void __cluster_dims__(kDraftCluster, 1, 1) __launch_bounds__(32 * WARPS, 512 / (16 * WARPS)) draft_verify_kernel(const DraftParams d) {
  constexpr int SEGS = kDraftCluster * WARPS, PER_LANE = SEGS / 32, THREADS = 32 * WARPS;
  __shared__ float2 sums[2][SEGS];  // one set a pass: the second pass never waits for readers of the first
  __shared__ float2 wsum[WARPS];
  __shared__ float2 before, target;
  __shared__ int first_out;         // first draft that is not kept
  __shared__ int found, win;        // drawn token; its segment
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  cluster_arrive_relaxed();
  const long long b = blockIdx.x / kDraftCluster;
  const int n = d.n_drafts ? min(max(d.n_drafts[b], 0), d.k) : d.k;
  if (tid == 0) {
    first_out = n;
    found = 0x7fffffff;
  }
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const long long x = d.drafts[b * d.k + i];
    bool keep = false;
    if (x >= 0 && x < d.V) {
      const float p = d.target[b * d.ts0 + i * d.ts1 + x];
      const float q = d.draft ? d.draft[b * d.ds0 + i * d.ds1 + x] : 1.f;
      // 24 x 24 bits: the product is exact in fp64
      keep = (double)d.accept_u[b * d.k + i] * (double)q < (double)p;
    }
    if (!keep) atomicMin(&first_out, i);
  }
  __syncthreads();
  const int a = first_out;
  const float* prow = d.target + b * d.ts0 + a * d.ts1;
  const float* qrow = (a < n && d.draft) ? d.draft + b * d.ds0 + a * d.ds1 : nullptr;
  // without draft probabilities the refused token itself has weight 0
  long long skip = (a < n && !d.draft) ? d.drafts[b * d.k + a] : -1;
  const int seg0 = (int)rank * WARPS + warp;
  const long long t0 = (long long)seg0 * d.seg, t1 = min(t0 + d.seg, (long long)d.V);
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float2 run = make_float2(0.f, 0.f);
    // eight values of each row a lane at a time, the next eight on their way meanwhile; behind the segment's end lanes
    // read its last value, with weight 0
    const int len = (int)(t1 - t0), skip_at = skip >= t0 && skip < t1 ? (int)(skip - t0) : -1;
    const float *pseg = prow + t0, *qseg = qrow ? qrow + t0 : nullptr;
    auto load = [&](int t, float (&p)[8], float (&q)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __ldcs(pseg + min(t + 32 * i, len - 1));
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = qseg ? __ldcs(qseg + min(t + 32 * i, len - 1)) : 0.f;
    };
    auto add = [&](int t, const float (&p)[8], const float (&q)[8]) {
      float2 eight;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float hi, lo, r;
        draft_weight(t + 32 * i == skip_at || t + 32 * i >= len ? 0.f : p[i], q[i], hi, lo);
        if (i == 0) {
          eight = make_float2(hi, lo);
        } else {
          two_sum(eight.x, hi, eight.x, r);
          eight.y = __fadd_rn(eight.y, __fadd_rn(r, lo));
        }
      }
      run = pair_add(run, eight);
    };
    if (len > 0) {
      float p0[8], q0[8], p1[8], q1[8];
      load(lane, p0, q0);
      for (int t = lane; t < len; t += 16 * 32) {
        if (t + 8 * 32 < len) load(t + 8 * 32, p1, q1);
        add(t, p0, q0);
        if (t + 8 * 32 >= len) break;
        if (t + 16 * 32 < len) load(t + 16 * 32, p0, q0);
        add(t + 8 * 32, p1, q1);
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1)
      run = pair_add(run, make_float2(__shfl_xor_sync(0xffffffffu, run.x, x), __shfl_xor_sync(0xffffffffu, run.y, x)));
    // a CTA's shared memory may be written from outside only once the CTA has begun: a small vocabulary leaves segments
    // empty, and their warps are here at once
    if (pass == 0) cluster_wait();
    if (lane < kDraftCluster) store_remote(&sums[pass][seg0], lane, run);
    cluster_sync();
    // the first warp of every CTA finds the segment of the drawn token
    if (warp == 0) {
      float2 v[PER_LANE], mine_sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) mine_sum = pair_add(mine_sum, v[i] = sums[pass][lane * PER_LANE + i]);
      const float2 incl = warp_scan(mine_sum, lane), total = shfl(incl, 31), want = pair_scale(total, d.sample_u[b]);
      float2 c = before_lane(incl, lane), mine_before = c;
      int mine = SEGS;
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) {
        const float2 next = pair_add(c, v[i]);
        if (mine == SEGS && v[i].x > 0.f && pair_above(next, want)) {
          mine = lane * PER_LANE + i;
          mine_before = c;
        }
        c = next;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, mine < SEGS);
      const int src = hit ? __ffs(hit) - 1 : 0;
      const int seg = __shfl_sync(0xffffffffu, mine, src);
      const float2 bef = shfl(mine_before, src);
      if (lane == 0) {
        win = hit ? seg : -1;
        before = bef;
        target = want;
      }
    }
    __syncthreads();
    // no weight over zero: the target's own row, once (the refused token counts again)
    if (win >= 0 || a == n) break;
    __syncthreads();
    qrow = nullptr;
    skip = -1;
  }
  // the CTA that holds the segment (or the first one, without any) answers
  const int w = win;
  if (w >= 0 ? (w / WARPS != (int)rank) : (rank != 0)) return;
  int token = -1;
  if (w >= 0) {
    // `per` consecutive values a thread, their sums scanned over the CTA
    const long long w0 = (long long)w * d.seg, w1 = min(w0 + d.seg, (long long)d.V);
    const int per = (int)((w1 - w0 + THREADS - 1) / THREADS);
    const long long a0 = w0 + (long long)tid * per, a1 = min(a0 + per, w1);
    float2 own = make_float2(0.f, 0.f);
    int last = -1;
    for (long long t = a0; t < a1; ++t) {
      float hi, lo;
      draft_weight(t == skip ? 0.f : prow[t], qrow ? qrow[t] : 0.f, hi, lo);
      if (hi > 0.f) last = (int)t;
      own = pair_add(own, make_float2(hi, lo));
    }
    const float2 incl = warp_scan(own, lane);
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    const float2 warps = warp_scan(lane < WARPS ? wsum[lane] : make_float2(0.f, 0.f), lane);
    const float2 base = warp ? shfl(warps, warp - 1) : make_float2(0.f, 0.f);
    float2 c = pair_add(pair_add(before, base), before_lane(incl, lane));
    for (long long t = a0; t < a1; ++t) {
      float hi, lo;
      draft_weight(t == skip ? 0.f : prow[t], qrow ? qrow[t] : 0.f, hi, lo);
      c = pair_add(c, make_float2(hi, lo));
      if (hi > 0.f && pair_above(c, target)) {
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
  for (int i = tid; i <= d.k; i += THREADS)
    d.tokens[b * (d.k + 1) + i] = i < a ? d.drafts[b * d.k + i] : i == a ? token : -1;
  if (tid == 0) {
    d.n_kept[b] = a;
    if (d.lengths) d.new_lengths[b] = d.lengths[b] - (n - a);
  }
}

// Memory of an argument (at NULL: none).
struct Range {
  const void* at;
  int64_t bytes;
};
static bool overlap(const Range& a, const Range& b) {
  const char *x = static_cast<const char*>(a.at), *y = static_cast<const char*>(b.at);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}
// Bytes from a table's first value to behind its last; false where that is more than 2^62.
static bool table_bytes(int64_t batch, int64_t rows, int64_t vocab, const int64_t* strides, int64_t* bytes) {
  int64_t a, b, n;
  if (__builtin_mul_overflow(batch - 1, strides[0], &a) || __builtin_mul_overflow(rows - 1, strides[1], &b) ||
      __builtin_add_overflow(a, b, &n) || __builtin_add_overflow(n, vocab, &n) || n > (1LL << 60))
    return false;
  *bytes = 4 * n;
  return true;
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
  if (target_strides[0] < 0 || target_strides[1] < 0 || (draft && (draft_strides[0] < 0 || draft_strides[1] < 0)))
    return fail(PALU_ERR_INVALID_ARG, "strides must not be negative");
  int64_t target_bytes, draft_bytes = 0;
  if (!table_bytes(batch, k + 1, vocab, target_strides, &target_bytes) ||
      (draft && !table_bytes(batch, k, vocab, draft_strides, &draft_bytes)))
    return fail(PALU_ERR_INVALID_ARG, "strides span more than the address space");
  // a sequence's answer must not overwrite what another has yet to read or has written
  const Range outs[3] = {{tokens, batch * (k + 1) * 8}, {n_kept, batch * 4}, {new_lengths, batch * 8}};
  const Range ins[7] = {{target, target_bytes}, {draft, draft_bytes}, {drafts, batch * k * 8}, {n_drafts, batch * 4},
                        {accept_u, batch * k * 4}, {sample_u, batch * 4}, {lengths, batch * 8}};
  for (int i = 0; i < 3; ++i) {
    for (const Range& in : ins) {
      // each sequence's element is read before its own is written
      const bool same = outs[i].at == in.at && ((i == 2 && in.at == lengths) || (i == 1 && in.at == n_drafts));
      if (overlap(outs[i], in) && !same) return fail(PALU_ERR_INVALID_ARG, "an output overlaps an input");
    }
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(PALU_ERR_INVALID_ARG, "outputs overlap each other");
  }
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Few sequences: more warps a CTA shorten the row's way.  Many: smaller CTAs, so that 64 sequences are one wave.
  const bool few = batch * kDraftCluster <= device_sm_count();
  const int segs = kDraftCluster * (few ? 16 : 8);
  p.seg = (int)((vocab + segs - 1) / segs);
  if (few)
    draft_verify_kernel<16><<<(unsigned)(batch * kDraftCluster), 512, 0, st>>>(p);
  else
    draft_verify_kernel<8><<<(unsigned)(batch * kDraftCluster), 256, 0, st>>>(p);
  return cuda_check(cudaGetLastError(), "draft_verify_kernel launch");
}
