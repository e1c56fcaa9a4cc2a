// Attention over the paged cache for few rows a KV head: single-token decode, a
// few drafted tokens.
//
// Bound by reading the cache: 512 bytes a token and KV head feed 4 * 128 * rows
// flops, far below the card's ratio for up to 16 rows.  So everything serves the
// loads: one persistent CTA an SM, a loading warp that keeps three 64 KB tiles
// (128 keys and values) in flight by TMA, one copy a page and 64-channel panel,
// and eight warps that take 16 tokens of each tile: scores as K q^T with the
// tokens as the m side and the rows as the n side of m16n8k16, so no product is
// spent on padding 3 or 7 rows to 16; a running maximum a warp, merged once a
// unit.  In fp16 the weights' reference lies 2^14 below the maximum: a warp may
// have 100,000 tokens whose weights next to a first token's 1 would be below the
// smallest fp16 number, and together count (304 sequences of 1,200,000: 12 times
// the bar of all roundings).
#pragma once

#include <math.h>

#include "paged_attn.cuh"
#include "splitk_attend.cuh"

namespace palu {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewStages = 3;
constexpr int kMergeStride = kHeadDim + 2;
template <bool BF16>
constexpr float kFewLift = BF16 ? 0.f : 14.f;  // log2: the largest weight; 2^14 < 65504

// One tile, as the loading warp hands it to the others.
struct TileMeta {
  UnitMeta u;
  int key0;         // place of the first key
  int valid;        // keys of the tile that exist (1 .. 128)
  int first, last;  // of the stretch
};
struct FewSmem {
  uint64_t full[kFewStages], empty[kFewStages], join;
  TileMeta meta[kFewStages];
  int failed;  // a wait ran out: the remaining ones are not begun
};
// tiles (1024-byte aligned), the warps' merge area (8 rows at a time), the rest
constexpr int kFewMergeBytes = kFewWarps * 8 * kMergeStride * 4;
constexpr int kFewSmemBytes = 1024 + kFewStages * 2 * kTileBytes + kFewMergeBytes + (int)sizeof(FewSmem);
static_assert(kFewSmemBytes + sizeof(PlanScratch) <= 232448, "shared memory of a few-rows CTA");

template <bool BF16>
__device__ __forceinline__ void mma_16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (BF16)
    mma_bf16(d, a0, a1, a2, a3, b0, b1);
  else
    mma_f16(d, a0, a1, a2, a3, b0, b1);
}

// What a CTA's stretch needs, set up by its first thread before all of them
// meet.
__device__ __forceinline__ uint8_t* few_smem(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
}
__device__ __forceinline__ FewSmem& few_shared(uint8_t* smem) {
  return *reinterpret_cast<FewSmem*>(smem + kFewStages * 2 * kTileBytes + kFewMergeBytes);
}
__device__ __forceinline__ void few_init(FewSmem& sh) {
  for (int i = 0; i < kFewStages; ++i) {
    mbar_init(&sh.full[i], 1);
    mbar_init(&sh.empty[i], kFewWarps);
    sh.meta[i] = TileMeta{};
  }
  mbar_init(&sh.join, kFewWarps);
  sh.failed = 0;
  fence_mbar_init();
}

// The stretch, by kFewThreads threads.  NT: n8 tiles of rows (8 or 16 rows a
// unit).
template <bool BF16, int NT, bool SPLIT>
__device__ __forceinline__ void few_stretch(const AttnParams& p, const PartSet& part, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                            const PlanScratch& plan, uint8_t* smem) {
  float* merge = reinterpret_cast<float*>(smem + kFewStages * 2 * kTileBytes);
  FewSmem& sh = few_shared(smem);
  constexpr int R = 8 * NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (plan.w1 > plan.w0) {
    if (warp == kFewWarps) {
      // ---- the loading warp
      unsigned bad = 0;
      int it = 0;
      // room for the next tile: all lanes go on or stop together
      auto room = [&] {
        if (it >= kFewStages)
          wait_or_fail(&sh.empty[it % kFewStages], ((it / kFewStages) - 1) & 1, &sh.failed, p.c.error);
        return !__any_sync(0xffffffffu, *(volatile int*)&sh.failed);
      };
      plan_walk<R, SPLIT>(p, part, &plan, [&](const UnitMeta& u) -> bool {
        if (lane < u.rows) {  // the unit's queries, to L2 while the tiles before it are worked on
          const uint16_t* q = row_query(p, u, lane);
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
        }
        for (int k = 0; k < u.n; ++k, ++it) {
          const int st = it % kFewStages, key0 = u.key0 + k * kKeyTile, valid = min(kKeyTile, u.key_end - key0);
          const int pages = (valid + p.c.page - 1) >> p.c.page_shift;
          const int page = lane < pages ? page_of(p, u.seq, key0 + lane * p.c.page, &bad) : 0;
          if (!room()) return false;
          if (lane == 0) {
            sh.meta[st] = TileMeta{u, key0, valid, k == 0, k == u.n - 1};
            mbar_arrive_expect_tx(&sh.full[st], pages * p.c.page * kHeadDim * 4);
          }
          __syncwarp();
          if (lane < pages) {
            const uint32_t kt = smem_addr(smem + st * 2 * kTileBytes) + lane * p.c.page * 128;
            tma_page(kt, &kmap, &sh.full[st], 0, u.kh, page);
            tma_page(kt + kPanelBytes, &kmap, &sh.full[st], 64, u.kh, page);
            tma_page(kt + kTileBytes, &vmap, &sh.full[st], 0, u.kh, page);
            tma_page(kt + kTileBytes + kPanelBytes, &vmap, &sh.full[st], 64, u.kh, page);
          }
        }
        return true;
      });
      const bool ended = room();
      if (ended && lane == 0) {  // a tile of no keys ends the line
        sh.meta[it % kFewStages].valid = 0;
        mbar_arrive(&sh.full[it % kFewStages]);
      }
      if (bad) atomicOr(p.c.error, bad);
      // no copy is in flight when the block ends, also where the others gave up (the stage that the end took had
      // been emptied)
      for (int k = max(it - kFewStages + (ended ? 1 : 0), 0); k < it; ++k)
        if (!mbar_wait_bounded(&sh.full[k % kFewStages], (k / kFewStages) & 1)) break;
    } else {
      // ---- 16 tokens of each tile a warp
      const int g = lane >> 2, c = lane & 3, mat = lane >> 3, rr = lane & 7, r0 = 16 * warp;
      float m_run[NT][2], l_run[NT][2], acc[NT][8][4];
      uint32_t qb[NT][8][2];
      int lim[NT][2];
      UnitMeta m = {};
      uint32_t joins = 0;
      // the eight warps meet (bounded, unlike a named barrier)
      auto join = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.join);
        wait_or_fail(&sh.join, joins & 1, &sh.failed, p.c.error);
        ++joins;
        __syncwarp();
      };
      for (int it = 0;; ++it) {
        const int st = it % kFewStages;
        wait_or_fail(&sh.full[st], (it / kFewStages) & 1, &sh.failed, p.c.error);
        if (__any_sync(0xffffffffu, *(volatile int*)&sh.failed)) break;
        const TileMeta& tm = sh.meta[st];
        const int valid = tm.valid, key0 = tm.key0, last = tm.last;
        if (valid == 0) break;
        if (tm.first) {
          m = tm.u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int rg = nt * 8 + g;
            const uint16_t* qh = row_query(p, m, rg);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              qb[nt][ks][0] = rg < m.rows ? *reinterpret_cast<const uint32_t*>(qh + 16 * ks + 2 * c) : 0u;
              qb[nt][ks][1] = rg < m.rows ? *reinterpret_cast<const uint32_t*>(qh + 16 * ks + 8 + 2 * c) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = nt * 8 + 2 * c + e;
              lim[nt][e] = r < m.rows ? unit_row_limit(p, plan, m, r) : 0;
              m_run[nt][e] = -INFINITY;
              l_run[nt][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
          }
        }
        const uint32_t kt = smem_addr(smem + st * 2 * kTileBytes), vt = kt + kTileBytes;
        if (r0 < valid) {
          if (valid < r0 + 16) {
            // whatever lies behind the last key must not reach the products: 0 * NaN is NaN
            const int z0 = valid - r0;
            for (int i = lane; i < (16 - z0) * 16; i += 32) {
              const uint32_t a = panel_addr(vt, r0 + z0 + (i >> 4), i & 15);
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          float sc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t a0, a1, a2, a3;
            ldsm_x4(a0, a1, a2, a3, panel_addr(kt, r0 + rr + ((mat & 1) << 3), 2 * ks + (mat >> 1)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16<BF16>(sc[nt], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
          }
          const int t = key0 + r0 + g;
          uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float* s = sc[nt];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[e] = t + 8 * (e >> 1) < lim[nt][e & 1] ? s[e] * p.scale_log2 : -INFINITY;
            float pr[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float bm = fmaxf(s[e], s[e + 2]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
              const float mn = fmaxf(m_run[nt][e], bm);
              const float top = mn == -INFINITY ? 0.f : mn;  // nothing seen so far: every weight is 0
              const float al = ex2f_(m_run[nt][e] - top), ref = top - kFewLift<BF16>;
              m_run[nt][e] = mn;
              pr[e] = ex2f_(s[e] - ref);
              pr[e + 2] = ex2f_(s[e + 2] - ref);
              l_run[nt][e] = l_run[nt][e] * al + (pr[e] + pr[e + 2]);
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                acc[nt][mt][e] *= al;
                acc[nt][mt][e + 2] *= al;
              }
            }
            // The weights enter as a rounded value and its remainder: two
            // products instead of one cost nothing here, and the output is
            // then as exact as its own rounding lets it be.
            const uint32_t h0 = pack2<BF16>(pr[0], pr[1]), h1 = pack2<BF16>(pr[2], pr[3]);
            const float2 f0 = unpack2<BF16>(h0), f1 = unpack2<BF16>(h1);
            ph[nt][0] = movmatrix_t(h0);
            ph[nt][1] = movmatrix_t(h1);
            pl[nt][0] = movmatrix_t(pack2<BF16>(pr[0] - f0.x, pr[1] - f0.y));
            pl[nt][1] = movmatrix_t(pack2<BF16>(pr[2] - f1.x, pr[3] - f1.y));
          }
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t a0, a1, a2, a3;
            ldsm_x4_t(a0, a1, a2, a3, panel_addr(vt, r0 + rr + ((mat >> 1) << 3), 2 * mt + (mat & 1)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16<BF16>(acc[nt][mt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              mma_16<BF16>(acc[nt][mt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
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
            float* mw = merge + warp * 8 * kMergeStride;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float l = l_run[nt][e];
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
              if (g == 0) {
                mw[(2 * c + e) * kMergeStride + kHeadDim] = m_run[nt][e];
                mw[(2 * c + e) * kMergeStride + kHeadDim + 1] = l;
              }
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mw[(2 * c + (e & 1)) * kMergeStride + 16 * mt + g + 8 * (e >> 1)] = acc[nt][mt][e];
            join();
            // a warp a row, four channels a lane
            const int r = nt * 8 + warp;
            if (r < m.rows) {
              const float* mr = merge + warp * kMergeStride;
              float M = -INFINITY;
#pragma unroll
              for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, mr[w * 8 * kMergeStride + kHeadDim]);
              const float ref = M == -INFINITY ? 0.f : M;
              float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int w = 0; w < kFewWarps; ++w) {
                const float* x = mr + w * 8 * kMergeStride;
                const float f = ex2f_(x[kHeadDim] - ref);
                L += x[kHeadDim + 1] * f;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] += x[4 * lane + i] * f;
              }
              const long long at = row_index(p, m, r);
              if (m.dest == kToOut) {
                const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
                uint2 v = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
                *reinterpret_cast<uint2*>(p.out + at * kHeadDim + 4 * lane) = v;
              } else {
                const long long rec = m.dest == kToRow ? (m.prefix ? 0 : (long long)p.N * p.Hq) + at
                                                       : (long long)m.dest * R + r;
                float2* ml = (m.dest == kToRow ? p.row_ml : part.ml) + rec;
                float* ac = (m.dest == kToRow ? p.row_acc : part.acc) + rec * kHeadDim;
                if (lane == 0) *ml = make_float2(M - kFewLift<BF16>, L);  // what the sums are relative to
                *reinterpret_cast<float4*>(ac + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        }
      }
    }
  }
}

}  // namespace palu
