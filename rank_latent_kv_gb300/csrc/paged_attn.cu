// Attention over the paged cache for few rows a KV head (single-token decode,
// a few drafted tokens), the joining of partial results, and the host side.
//
// paged_few_kernel is bound by reading the cache: 512 bytes a token and KV
// head feed 4 * 128 * rows flops, far below the card's ratio for up to 16
// rows.  So everything serves the loads: one persistent CTA an SM, a loading
// warp that keeps three 64 KB tiles (128 keys and values) in flight by TMA,
// one copy a page and 64-channel panel, and eight warps that take 16 tokens
// of each tile: scores as K q^T with the tokens as the m side and the rows as
// the n side of m16n8k16, so no product is spent on padding 3 or 7 rows to
// 16; a running maximum a warp, merged once a unit.  In fp16 the weights'
// reference lies 2^14 below the maximum: a warp may have 100,000 tokens whose
// weights next to a first token's 1 would be below the smallest fp16 number,
// and together count (304 sequences of 1,200,000: 36 times the bar of rounding).
#include <math.h>

#include <algorithm>

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
  PlanScratch plan;
  int failed;  // a wait ran out: the remaining ones are not begun
};
// tiles (1024-byte aligned), the warps' merge area (8 rows at a time), the rest
constexpr int kFewMergeBytes = kFewWarps * 8 * kMergeStride * 4;
constexpr int kFewSmemBytes = 1024 + kFewStages * 2 * kTileBytes + kFewMergeBytes + (int)sizeof(FewSmem);
static_assert(kFewSmemBytes <= 232448, "shared memory of paged_few_kernel");

template <bool BF16>
__device__ __forceinline__ void mma_16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (BF16)
    mma_bf16(d, a0, a1, a2, a3, b0, b1);
  else
    mma_f16(d, a0, a1, a2, a3, b0, b1);
}

// NT: n8 tiles of rows (8 or 16 rows a unit).
template <bool BF16, int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* merge = reinterpret_cast<float*>(smem + kFewStages * 2 * kTileBytes);
  FewSmem& sh = *reinterpret_cast<FewSmem*>(smem + kFewStages * 2 * kTileBytes + kFewMergeBytes);
  constexpr int R = 8 * NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_launch();
  if (tid == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kFewWarps);
      sh.meta[i] = TileMeta{};
    }
    mbar_init(&sh.join, kFewWarps);
    sh.failed = 0;
    fence_mbar_init();
  }
  plan_start<R, kFewThreads>(p, &sh.plan, tid);  // all threads meet in it
  if (sh.plan.w1 > sh.plan.w0) {
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
      plan_walk<R>(p, &sh.plan, [&](const UnitMeta& u) -> bool {
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
              lim[nt][e] = r < m.rows ? unit_row_limit(p, sh.plan, m, r) : 0;
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
                                                       : (long long)m.dest * p.part.R + r;
                float2* ml = (m.dest == kToRow ? p.row_ml : p.part.ml) + rec;
                float* ac = (m.dest == kToRow ? p.row_acc : p.part.acc) + rec * kHeadDim;
                if (lane == 0) *ml = make_float2(M - kFewLift<BF16>, L);  // what the sums are relative to
                *reinterpret_cast<float4*>(ac + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        }
      }
    }
  }
  // a launch before this one (the prefix on another kernel) has ended too when this one has
  grid_dep_wait();
}

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
struct JoinRowsParams {
  AttnParams a;
  PartSet prefix, own;
};

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
__device__ __forceinline__ void own_place(const JoinRowsParams& p, const SeqSpan& s, int b, int kh, int lr, long long* f,
                                          int* n, int* t) {
  const AttnParams& a = p.a;
  const int rt = lr / R, rows = min(R, s.n * a.Gq - rt * R);
  *n = own_tiles(s, rt * R, rows, a.Gq, a.S0);
  *t = LineCost<R>::tile(rows);
  *f = __ldcg(p.own.plan + 1 + b) + seq_ticks_warp<R>(s, rt, a.Gq, a.S0, a.c.kv_heads) + kh * unit_ticks<R>(rows, *n) +
       LineCost<R>::unit(rows);
}
template <int R>
__device__ __forceinline__ void prefix_place(const JoinRowsParams& p, int kh, int lr, long long* f, int* n, int* t) {
  const AttnParams& a = p.a;
  const int all_rows = a.N * a.Gq, rts = (all_rows + R - 1) / R, rt = lr / R;
  *n = prefix_tiles_of((int)__ldcg(p.prefix.plan + 1 + a.c.batch));
  const int rows = min(R, all_rows - rt * R);
  *t = LineCost<R>::tile(rows);
  *f = kh * prefix_ticks<R>(all_rows, rts, *n) + prefix_ticks<R>(all_rows, rt, *n) + LineCost<R>::unit(rows);
}

template <bool BF16, int STEP>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_rows_kernel(const JoinRowsParams p) {
  __shared__ JoinScratch sc;
  const AttnParams& a = p.a;
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
    if (p.own.R == 8) own_place<8>(p, s, b, kh, lr, &f, &n, &t);
    else if (p.own.R == 16) own_place<16>(p, s, b, kh, lr, &f, &n, &t);
    else own_place<kManyRows>(p, s, b, kh, lr, &f, &n, &t);
    w.own = parts(p.own, f, n, t, lr % p.own.R);
    if (p.prefix.R == 8) prefix_place<8>(p, kh, gr, &f, &n, &t);
    else if (p.prefix.R == 16) prefix_place<16>(p, kh, gr, &f, &n, &t);
    else prefix_place<kManyRows>(p, kh, gr, &f, &n, &t);
    w.pre = parts(p.prefix, f, n, t, gr % p.prefix.R);
  };
  Row w = find(row_first + (STEP > 1 ? warp : 0));
  grid_dep_wait();
  auto part = [&](int k, const float2*& ml, const float*& acc) {
    const bool pre = k < w.pre.n;
    const PartSet& ps = pre ? p.prefix : p.own;
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

constexpr int kOneLaunchKeys = 256;  // own keys a sequence up to which one launch takes them with a prefix of many rows

// Sizes that the host can know: which kernel takes the shared and which the
// own keys, and the workspace's parts.
struct AttnLayout {
  int grid_prefix, grid_own;
  bool shared;       // the prefix is a part of its own
  bool one_launch;   // both parts on the kernel for many rows
  int R_prefix, R_own;
  size_t plan_p, begun_p, ml_p, acc_p, plan_o, begun_o, ml_o, acc_o, row_ml, row_acc, total;
};

// SMs for the prefix where it and the own keys are two launches: they run side
// by side, each on SMs of its own, because a launch's beginning and end (about
// 25,000 and 10,000 clocks: its code has to be fetched) leave the memory idle.
// The own lengths are not known here: half of what the page table allows.
static int split_grid(const palu_paged_cache* c, int64_t all_rows, int32_t shared_pages, int R_prefix, int grid) {
  const int64_t t0 = prefix_tiles_of(shared_pages * c->page_size);
  const int64_t own = ((int64_t)(c->table_width - shared_pages) * c->page_size / 2 + kKeyTile - 1) / kKeyTile;
  const int64_t full = all_rows / R_prefix, rest = all_rows % R_prefix;
  double a;  // clocks of one SM
  if (R_prefix == kManyRows)
    a = c->kv_heads * (full * (20000. + 3100. * t0) + (rest > kManyRows / 2 ? 20000. + 3100. * t0 : rest ? 12500. + 2900. * t0 : 0.));
  else
    a = c->kv_heads * (5700. + 2900. * t0);
  const double b = (double)c->batch * c->kv_heads * (5700. + 2900. * own);
  int best = grid / 2;
  double least = INFINITY;
  for (int g = 1; g < grid; ++g) {
    const double t = std::max(25000. + a / g, 10000. + b / (grid - g));
    if (t < least) {
      least = t;
      best = g;
    }
  }
  return best;
}

// Whether reading the shared pages once pays.  It saves the tiles that the sequences would each read (a row tile each at
// least) beyond those of the whole batch's row tiles; it costs a second launch and, for every row, a record of each part
// that is written, read and joined.  28 heads of 4 KV heads, 512 own keys, bf16, read once and by each sequence: 16
// sequences of 1 token behind 1024 keys 19.1 and 14.3 us, behind 4096 23.3 and 33.0; 256 sequences of 5 behind 256 129 and
// 95 us, behind 4096 185 and 442; 16 of 1024 new tokens behind 8192 1901 and 1506 us.  In clocks, summed over the SMs:
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
  // Few own keys behind a prefix of many rows: one launch for both (256 rows behind 311,296 shared tokens and 1 own token
  // a sequence: 65 us in two launches, 55 in one; 96 rows behind 8192 and 580 own: 46 and 50).
  const bool few_keys = l->shared && l->R_prefix == kManyRows &&
                        (int64_t)(c->table_width - shared_pages) * c->page_size <= kOneLaunchKeys;
  l->R_own = few_keys ? kManyRows : R_rows;
  l->one_launch = l->shared && l->R_own == kManyRows;  // then the prefix has many rows, too
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
  const bool two = l->shared && !l->one_launch;
  const int grid = device_sm_count();
  l->grid_prefix = two && grid > 1 ? split_grid(c, all_rows, shared_pages, l->R_prefix, grid) : grid;
  l->grid_own = two && grid > 1 ? grid - l->grid_prefix : grid;
  // With shared pages the size is the same whether or not they are read once here: it also serves fewer tokens, and
  // any other number of them.
  const bool may_share = shared_pages > 0 && c->batch > 1;
  const size_t records = may_share ? 2 * (size_t)std::min(tokens, most_shared_tokens(c, q_heads)) * q_heads : 0;
  l->row_ml = take(records * sizeof(float2));
  l->row_acc = take(records * kHeadDim * sizeof(float));
  const size_t parts = o;
  take_parts(l->R_own, &l->plan_o, &l->begun_o, &l->ml_o, &l->acc_o);
  if (two) take_parts(l->R_prefix, &l->plan_p, &l->begun_p, &l->ml_p, &l->acc_p);
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

template <bool BF16>
static palu_status launch_few(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool dependent,
                              cudaStream_t s) {
  return p.part.R == 8 ? launch(paged_few_kernel<BF16, 1>, p.part.grid, kFewThreads, kFewSmemBytes, dependent, s,
                                "paged_few_kernel launch", p, km, vm)
                       : launch(paged_few_kernel<BF16, 2>, p.part.grid, kFewThreads, kFewSmemBytes, dependent, s,
                                "paged_few_kernel launch", p, km, vm);
}

// The launch of one part, on the kernel for its number of rows.  `dependent`:
// it may begin while the launch before it (the prefix) still runs.
static palu_status launch_part(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, bool dependent,
                               cudaStream_t s) {
  if (p.part.R == kManyRows) return launch_many(p, km, vm, bf16, s);
  return bf16 ? launch_few<true>(p, km, vm, dependent, s) : launch_few<false>(p, km, vm, dependent, s);
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
  const PartSet own = {reinterpret_cast<float2*>(ws + l.ml_o), reinterpret_cast<float*>(ws + l.acc_o),
                       reinterpret_cast<long long*>(ws + l.plan_o), reinterpret_cast<UnitMeta*>(ws + l.begun_o), l.grid_own,
                       l.R_own};
  const PartSet prefix = l.one_launch ? own
                                      : PartSet{reinterpret_cast<float2*>(ws + l.ml_p), reinterpret_cast<float*>(ws + l.acc_p),
                                                reinterpret_cast<long long*>(ws + l.plan_p), reinterpret_cast<UnitMeta*>(ws + l.begun_p),
                                                l.grid_prefix, l.R_prefix};
  const bool bf16 = cache->dtype == PALU_TYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (l.shared && !l.one_launch) {
    p.part = prefix;
    p.do_prefix = 1;
    if ((st = launch_part(p, km, vm, bf16, false, s)) != PALU_OK) return st;
  }
  p.part = own;
  p.do_prefix = l.one_launch;
  p.do_own = 1;
  if ((st = launch_part(p, km, vm, bf16, l.shared && !l.one_launch, s)) != PALU_OK) return st;
  if (!l.shared) {
    if (l.R_own < kManyRows) {
      const dim3 jgrid(l.grid_own, l.R_own);
      return bf16 ? launch(paged_join_units_kernel<true, 1>, jgrid, 32 * kJoinWarps, 0, true, s, "paged_join_units_kernel launch", p)
                  : launch(paged_join_units_kernel<false, 1>, jgrid, 32 * kJoinWarps, 0, true, s, "paged_join_units_kernel launch", p);
    }
    const dim3 jgrid(l.grid_own, l.R_own / kJoinWarps);
    return bf16 ? launch(paged_join_units_kernel<true, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                         "paged_join_units_kernel launch", p)
                : launch(paged_join_units_kernel<false, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                         "paged_join_units_kernel launch", p);
  }
  const JoinRowsParams jp = {p, prefix, own};
  const long long rows = (long long)p.N * p.Hq;
  if (rows <= kJoinRows)
    return bf16 ? launch(paged_join_rows_kernel<true, 1>, dim3((unsigned)rows), 32 * kJoinWarps, 0, true, s,
                         "paged_join_rows_kernel launch", jp)
                : launch(paged_join_rows_kernel<false, 1>, dim3((unsigned)rows), 32 * kJoinWarps, 0, true, s,
                         "paged_join_rows_kernel launch", jp);
  const dim3 jgrid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
  return bf16 ? launch(paged_join_rows_kernel<true, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                       "paged_join_rows_kernel launch", jp)
              : launch(paged_join_rows_kernel<false, kJoinWarps>, jgrid, 32 * kJoinWarps, 0, true, s,
                       "paged_join_rows_kernel launch", jp);
}
