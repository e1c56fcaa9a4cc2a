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
//   when a weight would pass 2^14: weights down to 2^-20 of the largest keep all
//   their bits.  The scales enter in units of 2^E, an E for each of the four
//   groups, which comes off again with the accumulators: the largest of a block
//   lies in 2^-3 .. 2, so that no p s passes 2^15 and, small scales or large, the
//   products keep all their bits down to 2^-17 of the largest weight's with the
//   largest scale of the block.  (E stops at -15: under scales of 2^-18 the units
//   are 2^-15.  Without units 65,536 tokens of scale 2^-14 behind a strong key were
//   off by 2^-6.  They cost 2 to 3 % of the time, one E for all groups 1 to 2 %.)
// A persistent CTA an SM; a loading warp copies 240 keys at a time, a page of a
// head by one bulk copy, into a ring of stages; 15 warps take a block of 16
// tokens of a stage each (for 9 to 16 rows, whose accumulators need the
// registers, 8 warps two blocks of 256 keys each: 87 us where 8 rows take 54).
//
// 16 sequences of up to 32,768 tokens, 28 heads of 4: 257 MB in 53.8 us, 9 of them
// fixed, then 5.7 TB/s; 64 of up to 8,191 with 16 heads of 16: 1,012 MB in 182 us.
// The copies alone take 48.7 and 161: instructions and memory bound it together
// (310 warp instructions a block, 50 % of the issue slots).
#pragma once

#include <math.h>

#include "paged4.cuh"
#include "paged_attn.cuh"
#include "splitk_attend.cuh"

namespace palu {

template <int NT>
constexpr int kFew4Warps = NT == 1 ? 15 : 8;
template <int NT>
constexpr int kFew4Threads = 32 * (kFew4Warps<NT> + 1);
template <int NT>
constexpr int kFew4Blocks = NT == 1 ? 15 : 16;                 // of a stage
template <int NT>
constexpr int kFew4StageBytes = kFew4Blocks<NT> * kBlock4;     // about 40 KB of codes, scales and zeros
constexpr int kFew4Stages = 4;
constexpr int kMerge4Stride = kHeadDim + 2;
template <int NT>
constexpr int kFew4MergeBytes = kFew4Warps<NT> * 8 * kMerge4Stride * 4;
constexpr float kLift4 = 6.f;      // log2: the reference's distance from the maximum
constexpr float kRaise4 = 14.f;    // log2: the largest weight before it is raised
constexpr float kNothing4 = -3e38f;  // a reference before any key has been seen: below any score

// One stage, as the loading warp hands it to the others.
struct Stage4Meta {
  int key0;         // place of the first key
  int valid;        // keys of the stage that exist; 0: the line has ended
  int first, last;  // of the stretch
  UnitMeta u;
};
struct Few4Smem {
  alignas(16) Stage4Meta meta[kFew4Stages];
  uint64_t full[kFew4Stages], empty[kFew4Stages], join;
  UnitMeta unit[16];           // each warp's, while it works on it
  int failed;                 // a wait ran out: the remaining ones are not begun
};
template <int NT>
constexpr int kFew4SmemBytes = 128 + kFew4Stages * kFew4StageBytes<NT> + kFew4MergeBytes<NT> + (int)sizeof(Few4Smem);
static_assert(kFew4SmemBytes<1> + sizeof(PlanScratch) <= 232448 && kFew4SmemBytes<2> + sizeof(PlanScratch) <= 232448,
              "shared memory of a few-rows CTA");

__device__ __forceinline__ uint8_t* few4_smem(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
}
template <int NT>
__device__ __forceinline__ Few4Smem& few4_shared(uint8_t* smem) {
  return *reinterpret_cast<Few4Smem*>(smem + kFew4Stages * kFew4StageBytes<NT> + kFew4MergeBytes<NT>);
}
template <int NT>
__device__ __forceinline__ void few4_init(Few4Smem& sh) {
  for (int i = 0; i < kFew4Stages; ++i) {
    mbar_init(&sh.full[i], 1);
    mbar_init(&sh.empty[i], kFew4Warps<NT>);
    sh.meta[i] = Stage4Meta{};
  }
  mbar_init(&sh.join, kFew4Warps<NT>);
  sh.failed = 0;
  fence_mbar_init();
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
// D = A(16x8) * B(8x8) in tf32
__device__ __forceinline__ void first_tf32(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A(16x16) * B(16x8) (+ D) in fp16, free to be moved
__device__ __forceinline__ void first_f16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void add_f16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
  const int e = query_shift(big);
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
  *factor = query_factor(e, p.scale_log2 * 0x1p24f);
}

// The stretch, by kFew4Threads<NT> threads: few4_work by the first kFew4Warps<NT>
// warps, few4_load by the one behind them.  NT: n8 tiles of rows (8 or 16 rows a
// unit).
template <int NT, bool SPLIT>
__device__ __forceinline__ void few4_load(const AttnParams& p, const PartSet& part, const PlanScratch& plan, uint8_t* smem) {
  constexpr int R = 8 * NT, kBlocks = kFew4Blocks<NT>, kStage = kFew4StageBytes<NT>;
  Few4Smem& sh = few4_shared<NT>(smem);
  const int lane = threadIdx.x & 31;
  if (plan.w1 <= plan.w0) return;
  unsigned bad = 0;
  int it = 0;
  // room for the next stage: all lanes go on or stop together
  auto room = [&] {
    if (it >= kFew4Stages)
      wait_or_fail(&sh.empty[it % kFew4Stages], ((it / kFew4Stages) - 1) & 1, &sh.failed, p.c.error);
    return !__any_sync(0xffffffffu, *(volatile int*)&sh.failed);
  };
  plan_walk<R, SPLIT, true>(p, part, &plan, [&](const UnitMeta& u) -> bool {
    if (lane < u.rows) {  // the unit's queries, to L2 while the tiles before it are worked on
      const uint16_t* q = row_query(p, u, lane);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
    }
    const int end = min(u.key0 + u.n * kKeyTile, u.key_end), per = p.c.page >> 4;
    // a stage's pages, one a lane: the blocks of each that it has
    struct Piece {
      int page, from, first, n;  // from: block of the page; first: block of the stage
    };
    auto lookup = [&](int key0) {
      const int b0 = key0 >> 4, b1 = min(b0 + kBlocks, (end + 15) >> 4), pi = (key0 >> p.c.page_shift) + lane;
      const int lo = max(b0, pi * per), hi = min(b1, (pi + 1) * per);
      Piece x = {0, lo - pi * per, lo - b0, hi - lo};
      if (x.n > 0) x.page = page_of(p, u.seq, lo << 4, &bad);
      return x;
    };
    Piece next = lookup(u.key0);
    for (int key0 = u.key0; key0 < end; key0 += 16 * kBlocks, ++it) {
      const int st = it % kFew4Stages, valid = min(16 * kBlocks, end - key0);
      const Piece x = next;
      next = lookup(key0 + 16 * kBlocks);  // in flight while this stage waits for room
      if (!room()) return false;
      if (lane == 0) {
        sh.meta[st] = Stage4Meta{key0, valid, key0 == u.key0, key0 + valid == end, u};
        mbar_arrive_expect_tx(&sh.full[st], ((valid + 15) >> 4) * kBlock4);
      }
      __syncwarp();
      if (x.n > 0)
        bulk_g2s(smem + st * kStage + x.first * kBlock4, page4(p.c, x.page, u.kh) + x.from * kBlock4, x.n * kBlock4, &sh.full[st]);
    }
    return true;
  });
  const bool ended = room();
  if (ended && lane == 0) {  // a stage of no keys ends the line
    sh.meta[it % kFew4Stages].valid = 0;
    mbar_arrive(&sh.full[it % kFew4Stages]);
  }
  if (bad) atomicOr(p.c.error, bad);
  // no copy is in flight when the block ends, also where the others gave up (the stage that the end took had
  // been emptied)
  for (int k = max(it - kFew4Stages + (ended ? 1 : 0), 0); k < it; ++k)
    if (!mbar_wait_bounded(&sh.full[k % kFew4Stages], (k / kFew4Stages) & 1)) break;
}

template <bool BF16, int NT>
__device__ __forceinline__ void few4_work(const AttnParams& p, const PartSet& part, const PlanScratch& plan, uint8_t* smem) {
  constexpr int R = 8 * NT, kWarps = kFew4Warps<NT>, kBlocks = kFew4Blocks<NT>, kStage = kFew4StageBytes<NT>;
  float* merge = reinterpret_cast<float*>(smem + kFew4Stages * kStage);
  Few4Smem& sh = few4_shared<NT>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (plan.w1 <= plan.w0) return;
  // ---- block `warp` of each stage (and `warp` + 8)
  const int g = lane >> 2, c = lane & 3;
  float ref[NT][2], acc[NT][8][4], zacc[NT][4], factor[NT][2];
  uint32_t qb[NT][4][4], qz[NT][2];
  int lim[NT][2], all_see = 0;  // tokens that every row of the unit sees
  uint32_t unit_inv[4];  // of the groups' scales: 2^-E, twice
  auto unit_log = [&](int j) { return 127 - (int)(__float_as_uint(half2_f(unit_inv[j]).x) >> 23); };  // E
  uint32_t joins = 0;
  // the warps meet (bounded, unlike a named barrier)
  auto join = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.join);
    wait_or_fail(&sh.join, joins & 1, &sh.failed, p.c.error);
    ++joins;
    __syncwarp();
  };
  // the zeros' product: rows 0 .. 3 are the groups, row 4, of ones, gives the weights' sum
  const uint32_t z_keep = g < 4 ? 0xffffffffu : 0u, z_ones = g == 4 ? 0x3c003c00u : 0u;
  for (uint32_t st = 0, turn = 0;;) {
    if (!__all_sync(0xffffffffu, mbar_try_wait(&sh.full[st], turn))) {
      wait_or_fail(&sh.full[st], turn, &sh.failed, p.c.error);
      if (__any_sync(0xffffffffu, *(volatile int*)&sh.failed)) break;
    }
    const uint4 head = lds128(smem_addr(&sh.meta[st]));
    const int key0 = (int)head.x, valid = (int)head.y;
    const bool last = head.w != 0;
    if (valid == 0) break;
    if (head.z) {
      const UnitMeta m = sh.meta[st].u;
      if (lane == 0) sh.unit[warp] = m;
      all_see = 0x7fffffff;
#pragma unroll
      for (int j = 0; j < 4; ++j) unit_inv[j] = 0x3c003c00u;  // anew, so that no unit's result depends on another's scales
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
          zacc[nt][e] = zacc[nt][e + 2] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
      }
      all_see = __reduce_min_sync(0xffffffffu, all_see);
    }
#pragma unroll 1
    for (int r0 = 16 * warp; r0 < min(valid, 16 * kBlocks); r0 += 16 * kWarps) {
      // a lane's codes lie 16 bytes a lane in a block, of the keys as of the values
      const uint32_t blk = smem_addr(smem) + st * kStage + (r0 >> 4) * kBlock4, codes = blk + 16 * lane;
      const uint32_t ks = blk + kKeyScales4 + 16 * g, vs = blk + kValueScales4 + 32 * c;
      // ---- scores
      float sc[NT][4];
      {
        const uint4 k0 = lds128(codes), k1 = lds128(codes + 512);
        const uint2 s0 = lds64(ks), s1 = lds64(ks + 128);
        const uint32_t z0 = __float_as_uint(lds_half(ks + 8 + 2 * c)), z1 = __float_as_uint(lds_half(ks + 136 + 2 * c));
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        const float2 f0a = half2_f(s0.x), f0b = half2_f(s0.y), f1a = half2_f(s1.x), f1b = half2_f(s1.y);
        const float f0[4] = {f0a.x, f0a.y, f0b.x, f0b.y}, f1[4] = {f1a.x, f1a.y, f1b.x, f1b.y};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) first_tf32(sc[nt], z0, z1, z0, z1, qz[nt][0], qz[nt][1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h0 = w0[j] >> 8, h1 = w1[j] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4];
            first_f16(d, w0[j] & kLow4, w1[j] & kLow4, w0[j] & kHigh4, w1[j] & kHigh4, qb[nt][j][0], qb[nt][j][1]);
            add_f16(d, h0 & kLow4, h1 & kLow4, h0 & kHigh4, h1 & kHigh4, qb[nt][j][2], qb[nt][j][3]);
            float* const s = sc[nt];
            s[0] = fmaf(f0[j], d[0], s[0]);
            s[1] = fmaf(f0[j], d[1], s[1]);
            s[2] = fmaf(f1[j], d[2], s[2]);
            s[3] = fmaf(f1[j], d[3], s[3]);
          }
        }
      }
      // ---- the values' scales
      const uint4 sa = lds128(vs), sb = lds128(vs + 16);  // tokens 2 c, 2 c + 1; 2 c + 8, 2 c + 9
      uint32_t s2[2][4] = {{sa.x, sa.y, sa.z, sa.w}, {sb.x, sb.y, sb.z, sb.w}};
      uint32_t z2[2] = {(lds32(vs + 128 + 4 * (g & 3)) & z_keep) | z_ones, (lds32(vs + 144 + 4 * (g & 3)) & z_keep) | z_ones};
      uint32_t bits = 0x30003000u;  // that a scale of 2^-3 .. 2 has
      if (__builtin_expect(key0 + r0 + 16 > min(all_see, key0 + valid), 0)) {
        // keys that some row does not see; what lies behind the last key must not reach the products: 0 * NaN is NaN
        const int left = valid - r0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t keep = (2 * c + 8 * i < left ? 0xffffu : 0u) | (2 * c + 8 * i + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
          for (int j = 0; j < 4; ++j) s2[i][j] &= keep;
          z2[i] &= keep;
          if (i == 0) bits &= keep;  // asked of a half-word only while its first token is there
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = g + 8 * i;
              if (at >= left || key0 + r0 + at >= lim[nt][e]) sc[nt][2 * i + e] = -INFINITY;
            }
        }
      }
      // in units: is a scale 2 or more, or a group's larger one of two tokens under 2^-3?  (By the bits: none is negative.)
      uint32_t su[2][4], top[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        su[0][j] = mul_f16x2(s2[0][j], unit_inv[j]);
        su[1][j] = mul_f16x2(s2[1][j], unit_inv[j]);
        top[j] = __vmaxu2(su[0][j], su[1][j]);
      }
      const uint32_t any = top[0] | top[1] | top[2] | top[3], all = top[0] & top[1] & top[2] & top[3];
      // ---- weights; and is one above its bound?
      float x[NT][4], over = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[nt][e] = fmaf(sc[nt][e], factor[nt][e & 1], -ref[nt][e & 1]);
          over = fmaxf(over, x[nt][e]);
        }
      if (__builtin_expect(__any_sync(0xffffffffu, ((any & 0x40004000u) | (~all & bits)) != 0 || over > kRaise4), 0)) {
        // other units for a group whose largest scale of the block is not in their range
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = __vmaxu2(s2[0][j], s2[1][j]);
          const unsigned largest = __reduce_max_sync(0xffffffffu, max(x & 0x7fffu, x >> 16 & 0x7fffu));
          // the scale is 2^at times 1/2 .. 1
          const int at = (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)largest))) >> 23) - 126;
          const int to = min(max(at, -15), 16), from = unit_log(j);  // (at most 16, whatever is not finite)
          if (largest != 0 && (at > from + 1 || (at < from - 2 && to != from))) {
            const float f = __uint_as_float((uint32_t)(127 + from - to) << 23), inv = __uint_as_float((uint32_t)(127 - to) << 23);
            unit_inv[j] = pack_f16x2(inv, inv);
            su[0][j] = mul_f16x2(s2[0][j], unit_inv[j]);
            su[1][j] = mul_f16x2(s2[1][j], unit_inv[j]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                acc[nt][2 * j][e] *= f;
                acc[nt][2 * j + 1][e] *= f;
              }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the scores themselves: next to a reference that says "nothing yet" they were lost
            x[nt][e] = sc[nt][e] * factor[nt][e];
            x[nt][e + 2] = sc[nt][e + 2] * factor[nt][e];
            float bm = fmaxf(x[nt][e], x[nt][e + 2]);
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, i));
            const float to = bm > ref[nt][e] + kRaise4 ? bm - kLift4 : ref[nt][e], al = ex2f_(ref[nt][e] - to);
            ref[nt][e] = to;
            zacc[nt][e] *= al;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              acc[nt][mt][e] *= al;
              acc[nt][mt][e + 2] *= al;
            }
            x[nt][e] -= to;
            x[nt][e + 2] -= to;
          }
      }
      uint32_t ph[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        ph[nt][0] = movmatrix_t(pack_f16x2(ex2f_(x[nt][0]), ex2f_(x[nt][1])));
        ph[nt][1] = movmatrix_t(pack_f16x2(ex2f_(x[nt][2]), ex2f_(x[nt][3])));
        add_f16(zacc[nt], z2[0], 0u, z2[1], 0u, ph[nt][0], ph[nt][1]);
      }
      // ---- values
      const uint4 v0 = lds128(codes + kValueCodes4), v1 = lds128(codes + kValueCodes4 + 512);
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          b[nt][0] = mul_f16x2(ph[nt][0], su[0][j]);
          b[nt][1] = mul_f16x2(ph[nt][1], su[1][j]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = w[2 * j + i], y = x >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            add_f16(acc[nt][2 * j + i], x & kLow4, x & kHigh4, y & kLow4, y & kHigh4, b[nt][0], b[nt][1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[st]);
    if (++st == kFew4Stages) {
      st = 0;
      turn ^= 1;
    }
    if (last) {
      const UnitMeta& m = sh.unit[warp];
      // join the warps' states, 8 rows at a time, and write the unit's result
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        join();
        float* mw = merge + warp * 8 * kMerge4Stride;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float l = __shfl_sync(0xffffffffu, zacc[nt][e], 4 * 4 + c);
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
            const float up = __uint_as_float((uint32_t)(127 + unit_log(mt >> 1)) << 23);
            to[0] = fmaf(acc[nt][mt][e], up * 0x1p24f, z);
            to[8] = fmaf(acc[nt][mt][e + 2], up * 0x1p20f, z);
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
