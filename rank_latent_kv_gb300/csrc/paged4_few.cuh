// Attention over the 4-bit paged cache for few rows a KV head: single-token
// decode, a few drafted tokens.
//
// 160 bytes a token and KV head where fp16 pages have 512, so the instructions
// between the bytes and the products are what has to be few: at memory speed an
// SM has 110 clocks for 16 tokens.  So the codes go into m16n8k16 products as
// they are.  Four bits under a mask, in the low bits of an fp16 number, are the
// subnormal c 2^-24 (or, masked four bits higher, 16 c 2^-24), which the tensor
// cores take exactly: one operation for two codes, no conversion.  The blocks
// of the pages hold the codes in the order in which a lane needs them.
//   Scores: tokens are the m side, rows the n side, as in paged_few.cuh.
//   s q^T c over the 32 channels of a group is one accumulator, multiplied by
//   the tokens' fp32 scales as it is added to the others; the zeros' part, the
//   sum over groups of z (sum of q), is one tf32 product with the sums of q
//   split in two.  q enters in fp16 times a power of two that brings its row's
//   largest value to 2^13 .. 2^14 (and its pairs under the higher mask another
//   2^-4), so that bf16's range does not matter.
//   Values: a row's weights p, in fp16, are the n side of the products with the
//   zeros and, times the tokens' scales of the group, with the codes.  p is
//   relative to a reference that lies 2^6 under the row's maximum and is raised
//   when a weight would pass 2^14; where a scale above 1 is met both bounds are
//   lowered by its power of two, so that no p s passes 2^15.  Weights down to
//   2^-20 of the largest keep all their bits.
// A persistent CTA an SM; a loading warp copies a tile's blocks, a page of a
// head by one bulk copy, into a ring of stages; the other warps take a block
// of 16 tokens of a tile each, in two groups that take tiles in turn (one group
// for 9 to 16 rows, whose accumulators need the registers).
#pragma once

#include <math.h>

#include "paged4.cuh"
#include "paged_attn.cuh"
#include "splitk_attend.cuh"

namespace palu {

constexpr int kTile4 = kKeyTile / 16 * kBlock4;  // 20 KB of codes, scales and zeros
template <int NT>
constexpr int kFew4Warps = NT == 1 ? 16 : 8;
template <int NT>
constexpr int kFew4Threads = 32 * (kFew4Warps<NT> + 1);
constexpr int kMerge4Stride = kHeadDim + 2;
template <int NT>
constexpr int kFew4MergeBytes = kFew4Warps<NT> * 8 * kMerge4Stride * 4;
template <int NT>
constexpr int kFew4Stages = NT == 1 ? 7 : 9;
constexpr float kLift4 = 6.f;      // log2: the reference's distance from the maximum
constexpr float kRaise4 = 14.f;    // log2: the largest weight before it is raised
constexpr float kNothing4 = -1e30f;  // a reference before any key has been seen

// One tile, as the loading warp hands it to the others.
struct Tile4Meta {
  UnitMeta u;
  int key0;         // place of the first key
  int valid;        // keys of the tile that exist (1 .. 128); 0: the line has ended
  int first, last;  // of the stretch
};
template <int NT>
struct Few4Smem {
  uint64_t full[kFew4Stages<NT>], empty[kFew4Stages<NT>], join;
  Tile4Meta meta[kFew4Stages<NT>];
  int failed;  // a wait ran out: the remaining ones are not begun
};
template <int NT>
constexpr int kFew4SmemBytes = 128 + kFew4Stages<NT> * kTile4 + kFew4MergeBytes<NT> + (int)sizeof(Few4Smem<NT>);
static_assert(kFew4SmemBytes<1> + sizeof(PlanScratch) <= 232448 && kFew4SmemBytes<2> + sizeof(PlanScratch) <= 232448,
              "shared memory of a few-rows CTA");

__device__ __forceinline__ uint8_t* few4_smem(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
}
template <int NT>
__device__ __forceinline__ Few4Smem<NT>& few4_shared(uint8_t* smem) {
  return *reinterpret_cast<Few4Smem<NT>*>(smem + kFew4Stages<NT> * kTile4 + kFew4MergeBytes<NT>);
}
template <int NT>
__device__ __forceinline__ void few4_init(Few4Smem<NT>& sh) {
  for (int i = 0; i < kFew4Stages<NT>; ++i) {
    mbar_init(&sh.full[i], 1);
    mbar_init(&sh.empty[i], kFew4Warps<NT>);
    sh.meta[i] = Tile4Meta{};
  }
  mbar_init(&sh.join, kFew4Warps<NT>);
  sh.failed = 0;
  fence_mbar_init();
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
__device__ __forceinline__ float lds_half(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// D = A(16x8) * B(8x8) + D in tf32
__device__ __forceinline__ void mma_tf32(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 half2_f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

constexpr uint32_t kLow4 = 0x000f000fu, kHigh4 = 0x00f000f0u;  // codes as c 2^-24 and 16 c 2^-24

// A row's queries as a lane's side of the products: channels 8 c .. 8 c + 7 of
// each group, times 2^e.  `factor`: what takes the scores back to log2.
template <bool BF16>
__device__ __forceinline__ void few4_queries(const AttnParams& p, const uint16_t* q, bool there, int c, uint32_t (&qb)[4][4],
                                             uint32_t (&qz)[2], float* factor) {
  uint4 raw[4];
  float big = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    raw[j] = there ? __ldg(reinterpret_cast<const uint4*>(q + 32 * j + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t r[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(r[i]);
      big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  }
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
  // 2^e with big 2^e in [2^13, 2^14); rows of zeros or of infinities as they are
  const int ex = (int)(__float_as_uint(big) >> 23);
  const int e = ex == 0 || ex == 255 ? 0 : max(min(13 + 127 - ex, 100), -113);
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
  float mine = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t r[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = unpack2<BF16>(r[i]);
      f.x *= up;
      f.y *= up;
      sum += f.x + f.y;
      const float m = i & 1 ? 0.0625f : 1.f;
      qb[j][i] = pack_f16x2(f.x * m, f.y * m);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (j == c) mine = sum;
  }
  mine *= 0x1p-24f;
  qz[0] = to_tf32(mine);
  qz[1] = to_tf32(mine - __uint_as_float(qz[0]));
  *factor = __uint_as_float((uint32_t)(127 - e) << 23) * (p.scale_log2 * 0x1p24f);
}

// The stretch, by kFew4Threads<NT> threads.  NT: n8 tiles of rows (8 or 16 rows
// a unit).
template <bool BF16, int NT, bool SPLIT>
__device__ __forceinline__ void few4_stretch(const AttnParams& p, const PartSet& part, const PlanScratch& plan, uint8_t* smem) {
  constexpr int kWarps = kFew4Warps<NT>, kStages = kFew4Stages<NT>, kGroups = kWarps / 8, R = 8 * NT;
  float* merge = reinterpret_cast<float*>(smem + kStages * kTile4);
  Few4Smem<NT>& sh = few4_shared<NT>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (plan.w1 <= plan.w0) return;
  if (warp == kWarps) {
    // ---- the loading warp
    unsigned bad = 0;
    int it = 0;
    // room for the next tile: all lanes go on or stop together
    auto room = [&] {
      if (it >= kStages) wait_or_fail(&sh.empty[it % kStages], ((it / kStages) - 1) & 1, &sh.failed, p.c.error);
      return !__any_sync(0xffffffffu, *(volatile int*)&sh.failed);
    };
    plan_walk<R, SPLIT, true>(p, part, &plan, [&](const UnitMeta& u) -> bool {
      if (lane < u.rows) {  // the unit's queries, to L2 while the tiles before it are worked on
        const uint16_t* q = row_query(p, u, lane);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
      }
      for (int k = 0; k < u.n; ++k, ++it) {
        const int st = it % kStages, key0 = u.key0 + k * kKeyTile, valid = min(kKeyTile, u.key_end - key0);
        const int pages = (valid + p.c.page - 1) >> p.c.page_shift, blocks = (valid + 15) >> 4, per = p.c.page >> 4;
        const int page = lane < pages ? page_of(p, u.seq, key0 + lane * p.c.page, &bad) : 0;
        if (!room()) return false;
        if (lane == 0) {
          sh.meta[st] = Tile4Meta{u, key0, valid, k == 0, k == u.n - 1};
          mbar_arrive_expect_tx(&sh.full[st], blocks * kBlock4);
        }
        __syncwarp();
        if (lane < pages)
          bulk_g2s(smem + st * kTile4 + lane * per * kBlock4, page4(p.c, page, u.kh), min(per, blocks - lane * per) * kBlock4,
                   &sh.full[st]);
      }
      return true;
    });
    const bool ended = room();
    if (ended && lane == 0) {  // a tile of no keys ends the line
      sh.meta[it % kStages].valid = 0;
      mbar_arrive(&sh.full[it % kStages]);
    }
    if (bad) atomicOr(p.c.error, bad);
    // no copy is in flight when the block ends, also where the others gave up (the stage that the end took had
    // been emptied)
    for (int k = max(it - kStages + (ended ? 1 : 0), 0); k < it; ++k)
      if (!mbar_wait_bounded(&sh.full[k % kStages], (k / kStages) & 1)) break;
    return;
  }
  // ---- 16 tokens of each tile of its group a warp
  const int g = lane >> 2, c = lane & 3, group = warp >> 3, r0 = 16 * (warp & 7);
  float ref[NT][2], l_run[NT][2], acc[NT][8][4], zacc[NT][4], factor[NT][2];
  uint32_t qb[NT][4][4], qz[NT][2];
  int lim[NT][2], all_see = 0;  // tokens that every row of the unit sees
  UnitMeta m = {};
  uint32_t joins = 0;
  // the warps meet (bounded, unlike a named barrier)
  auto join = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.join);
    wait_or_fail(&sh.join, joins & 1, &sh.failed, p.c.error);
    ++joins;
    __syncwarp();
  };
  for (int it = 0;; ++it) {
    const int st = it % kStages;
    wait_or_fail(&sh.full[st], (it / kStages) & 1, &sh.failed, p.c.error);
    if (__any_sync(0xffffffffu, *(volatile int*)&sh.failed)) break;
    const Tile4Meta& tm = sh.meta[st];
    const int valid = tm.valid, key0 = tm.key0, last = tm.last;
    if (valid == 0) break;
    if (tm.first) {
      m = tm.u;
      all_see = 0x7fffffff;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int rg = nt * 8 + g;
        float f;
        few4_queries<BF16>(p, row_query(p, m, rg), rg < m.rows, c, qb[nt], qz[nt], &f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * c + e;
          factor[nt][e] = __shfl_sync(0xffffffffu, f, (2 * c + e) * 4);
          lim[nt][e] = r < m.rows ? unit_row_limit(p, plan, m, r) : 0;
          all_see = r < m.rows ? min(all_see, lim[nt][e]) : all_see;
          ref[nt][e] = kNothing4;
          l_run[nt][e] = 0.f;
          zacc[nt][e] = zacc[nt][e + 2] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
      }
      all_see = __reduce_min_sync(0xffffffffu, all_see);
    }
    if (it % kGroups == group && r0 < valid) {
      const uint32_t blk = smem_addr(smem + st * kTile4) + (warp & 7) * kBlock4;
      // ---- scores
      const uint4 k0 = lds128(blk + 64 * g + 16 * c), k1 = lds128(blk + 64 * (g + 8) + 16 * c);
      const uint2 s0 = lds64(blk + kKeyScales4 + 16 * g), s1 = lds64(blk + kKeyScales4 + 16 * (g + 8));
      const uint32_t z0 = __float_as_uint(lds_half(blk + kKeyScales4 + 16 * g + 8 + 2 * c));
      const uint32_t z1 = __float_as_uint(lds_half(blk + kKeyScales4 + 16 * (g + 8) + 8 + 2 * c));
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
      const float2 f0a = half2_f(s0.x), f0b = half2_f(s0.y), f1a = half2_f(s1.x), f1b = half2_f(s1.y);
      const float f0[4] = {f0a.x, f0a.y, f0b.x, f0b.y}, f1[4] = {f1a.x, f1a.y, f1b.x, f1b.y};
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        mma_tf32(sc[nt], z0, z1, z0, z1, qz[nt][0], qz[nt][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t h0 = w0[j] >> 8, h1 = w1[j] >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(d, w0[j] & kLow4, w1[j] & kLow4, w0[j] & kHigh4, w1[j] & kHigh4, qb[nt][j][0], qb[nt][j][1]);
          mma_f16(d, h0 & kLow4, h1 & kLow4, h0 & kHigh4, h1 & kHigh4, qb[nt][j][2], qb[nt][j][3]);
          sc[nt][0] = fmaf(f0[j], d[0], sc[nt][0]);
          sc[nt][1] = fmaf(f0[j], d[1], sc[nt][1]);
          sc[nt][2] = fmaf(f1[j], d[2], sc[nt][2]);
          sc[nt][3] = fmaf(f1[j], d[3], sc[nt][3]);
        }
      }
      // ---- the values' scales, and how far they leave room for the weights
      const uint32_t vb = blk + kValueCodes4, vs = blk + kValueScales4 + 32 * c;
      const uint4 sa = lds128(vs), sb = lds128(vs + 16);  // tokens 2 c, 2 c + 1; 2 c + 8, 2 c + 9
      uint32_t s2[2][4] = {{sa.x, sa.y, sa.z, sa.w}, {sb.x, sb.y, sb.z, sb.w}};
      uint32_t z2[2] = {0u, 0u};
      if (g < 4) {
        z2[0] = lds32(vs + 128 + 4 * g);
        z2[1] = lds32(vs + 128 + 16 + 4 * g);
      }
      const int t0 = key0 + r0;
      const bool cut = t0 + 16 > all_see;
      if (cut) {
        // what lies behind the last key must not reach the products: 0 * NaN is NaN
        const int left = valid - r0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t keep = (2 * c + 8 * h < left ? 0xffffu : 0u) | (2 * c + 8 * h + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
          for (int j = 0; j < 4; ++j) s2[h][j] &= keep;
          z2[h] &= keep;
        }
      }
      uint32_t smax = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) smax = max_u16x2(smax, max_u16x2(s2[0][j], s2[1][j]));
      float high = kRaise4;  // the largest weight, log2
      if (__any_sync(0xffffffffu, (smax & 0xffffu) > 0x3c00u || (smax >> 16) > 0x3c00u)) {
        const uint32_t x = __reduce_max_sync(0xffffffffu, max(smax & 0xffffu, smax >> 16));
        high = kRaise4 - (float)(min((int)(x >> 10), 30) - 14);  // below 2^(exponent + 1)
      }
      const float lift = kLift4 - (kRaise4 - high);
      // ---- weights
      uint32_t ph[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* s = sc[nt];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= factor[nt][e & 1];
        if (cut)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = t0 + g + 8 * (e >> 1) < lim[nt][e & 1] ? s[e] : -INFINITY;
        const bool over = fmaxf(s[0], s[2]) > ref[nt][0] + high || fmaxf(s[1], s[3]) > ref[nt][1] + high;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float bm = fmaxf(s[e], s[e + 2]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
            const float to = bm > ref[nt][e] + high ? bm - lift : ref[nt][e], al = ex2f_(ref[nt][e] - to);
            ref[nt][e] = to;
            l_run[nt][e] *= al;
            zacc[nt][e] *= al;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              acc[nt][mt][e] *= al;
              acc[nt][mt][e + 2] *= al;
            }
          }
        }
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2f_(s[e] - ref[nt][e & 1]);
        l_run[nt][0] += pr[0] + pr[2];
        l_run[nt][1] += pr[1] + pr[3];
        ph[nt][0] = movmatrix_t(pack_f16x2(pr[0], pr[1]));
        ph[nt][1] = movmatrix_t(pack_f16x2(pr[2], pr[3]));
        mma_f16(zacc[nt], z2[0], 0u, z2[1], 0u, ph[nt][0], ph[nt][1]);
      }
      // ---- values
      const uint4 v0 = lds128(vb + 16 * lane), v1 = lds128(vb + 512 + 16 * lane);
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          b[nt][0] = mul_f16x2(ph[nt][0], s2[0][j]);
          b[nt][1] = mul_f16x2(ph[nt][1], s2[1][j]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = w[2 * j + h], y = x >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(acc[nt][2 * j + h], x & kLow4, x & kHigh4, y & kLow4, y & kHigh4, b[nt][0], b[nt][1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[st]);
    if (last) {
      // join the warps' states, 8 rows at a time, and write the unit's result
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        join();
        float* mw = merge + warp * 8 * kMerge4Stride;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = l_run[nt][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
          if (g == 0) {
            mw[(2 * c + e) * kMerge4Stride + kHeadDim] = ref[nt][e] == kNothing4 ? -INFINITY : ref[nt][e];
            mw[(2 * c + e) * kMerge4Stride + kHeadDim + 1] = l;
          }
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = __shfl_sync(0xffffffffu, zacc[nt][e], (mt >> 1) * 4 + c);
            float* to = mw + (2 * c + e) * kMerge4Stride + 16 * mt + g;
            to[0] = fmaf(acc[nt][mt][e], 0x1p24f, z);
            to[8] = fmaf(acc[nt][mt][e + 2], 0x1p20f, z);
          }
        join();
        // a warp a row, four channels a lane
        const int r = nt * 8 + warp;
        if (warp < 8 && r < m.rows) {
          const float* mr = merge + warp * kMerge4Stride;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mr[w * 8 * kMerge4Stride + kHeadDim]);
          const float base = M == -INFINITY ? 0.f : M;
          float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float* x = mr + w * 8 * kMerge4Stride;
            const float f = ex2f_(x[kHeadDim] - base);
            L += x[kHeadDim + 1] * f;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += x[4 * lane + i] * f;
          }
          const long long at = row_index(p, m, r);
          if (m.dest == kToOut) {
            const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
            *reinterpret_cast<uint2*>(p.out + at * kHeadDim + 4 * lane) =
                make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
          } else {
            const long long rec = m.dest == kToRow ? (m.prefix ? 0 : (long long)p.N * p.Hq) + at : (long long)m.dest * R + r;
            float2* ml = (m.dest == kToRow ? p.row_ml : part.ml) + rec;
            float* ac = (m.dest == kToRow ? p.row_acc : part.acc) + rec * kHeadDim;
            if (lane == 0) *ml = make_float2(M, L);
            *reinterpret_cast<float4*>(ac + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
  }
}

}  // namespace palu
