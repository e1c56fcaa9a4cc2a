// Attention over the paged cache for many rows a KV head: a shared prefix
// that all sequences' queries read, several drafted tokens, prompt chunks.
//
// From about 300 rows on, the 4 * 128 flops a (row, key) cost more than
// reading the key: the tensor cores are the bound, and 128 rows against 128
// keys (two products of 128^3) take 1024 clocks of them, in which the
// softmax's 16,384 exponentials have to be done too.  One persistent CTA an
// SM works on 256 rows at a time, as two row halves of 128 that take turns:
// while one half's weights are computed by its 128 threads (a row a thread, no
// shuffles), the tensor cores work for the other.  Both halves use the same
// keys and values, so a tile is read once for 256 rows.  A unit of at most
// 128 rows gives its even tiles to one half and its odd tiles to the other, and
// the two results are joined at the end.
//
//   TMEM (512 columns): S0 S1 O0 O1, 128 fp32 columns each.  The weights P
//   overwrite their scores as 16-bit pairs and enter the second product from
//   there, 64 keys as soon as they are ready, so that a half's exponentials
//   overlap with its product.  (Two score buffers of 64 keys a half gain
//   nothing: a product 128 x 64 x 16 from shared memory takes the 64 clocks of
//   one 128 x 128 x 16; measured 3,950 clocks a tile pair.)
//   A tile pair takes about 3,100 clocks: the products alone 2,048, in which
//   they read 192 KB of shared memory and the copies write 64, at 128 bytes a
//   clock as long again.  1,024 tokens of 8 heads over 53,248 keys: 160 us,
//   1383 TFLOP/s.
//   Shared memory: Q0 Q1 (32 KB each), a ring of five 32 KB tiles that holds
//   K and V of successive key tiles in turn.
//   Warps 0-3, 4-7: the halves' softmax; warp 8: loads; warps 9, 10: the
//   halves' products.  (The tensor cores take a product only when they are
//   nearly done with those before it, so a warp that issues for both halves
//   leaves them idle whenever it waits: 3,250 clocks a tile pair.)
//
// The reference of the weights is raised only when the maximum grows by more
// than 2^8: the accumulator in TMEM is rescaled a few times a unit instead of
// once a tile.  In fp16 it lies 2^6 below the maximum, so that weights reach
// 2^14 at most and those down to 2^-20 of the largest keep all their bits.  Weights are rounded
// once, to the type of the values (the tensor cores take no other); their sum is
// kept in fp32 before that rounding, so the roundings' errors average out
// instead of adding up.
#pragma once

#include "paged_attn.cuh"
#include "splitk_attend.cuh"

namespace palu {

constexpr int kManyThreads = 352;
constexpr int kRing = 5;
// Two arrival barriers a ring slot, used in turn: where the halves have tiles of their own, one may ask for an item
// while the slot's item before it, the other half's, is still on its way, and one barrier's parity could not tell the
// two apart.
constexpr int kFull = 2 * kRing;
constexpr int kHalf = 128;
constexpr int kStageBytes = 32 * 36 * 4;  // 128 bytes of a warp's 32 rows, padded against bank conflicts

struct ManySmem {
  uint64_t kv_full[kFull], kv_empty[kRing];
  uint64_t meta_full[2], meta_empty[2];
  uint64_t q_full, s_full[2], p_full[2][2], unit_done, join, drain[2], token[2];
  UnitMeta meta[2];
  uint32_t tmem;
  int failed;
};
constexpr int kManySmemBytes = 1024 + (2 + kRing) * kTileBytes + (int)sizeof(ManySmem);
static_assert(kManySmemBytes + sizeof(PlanScratch) <= 232448, "shared memory of a many-rows CTA");

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_alloc(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(dst)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t t) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One lane of a converged warp.  Products and commits are issued under it by a warp whose control flow is uniform:
// under a branch on the lane number the compiler has to assume several lanes, and a product took 110 clocks to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// d (+)= a b, both operands in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// d (+)= a b, a in TMEM
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// 32 columns of this warp's 32 lanes, a lane a thread
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The loads before it have arrived: r passes through, so that nothing that uses it moves in front.
__device__ __forceinline__ void tc_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
  tc_wait_ld16(r);
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: byte offsets between
// 8-row groups (stride) and, for an operand whose rows run along N (the
// values: 64 channels a panel), between panels (lead).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ULL << 46 | 2ULL << 61;
}
// Instruction descriptor: fp32 accumulator, 128 x 128, both operands of one 16-bit type.
template <bool BF16>
__device__ constexpr uint32_t instr_desc(bool b_n_major) {
  return 1u << 4 | (BF16 ? 1u << 7 | 1u << 10 : 0u) | (b_n_major ? 1u << 16 : 0u) | (128u >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fma2(float& x, float& y, float s, float c) {  // (x, y) <- (x, y) s + c
  uint64_t v, ss, cc;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
  asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(ss), "l"(cc));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ void add2(float& ax, float& ay, float x, float y) {
  uint64_t a, v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(ax), "f"(ay));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(v));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(ax), "=f"(ay) : "l"(a));
}

constexpr float kRaise = 8.f;  // log2 of how far the maximum may grow before the reference is raised

__device__ __forceinline__ uint8_t* many_smem(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
}

// The CTA's stretch, by all kManyThreads threads; `start` is run by warps 8 to
// 10 before the others may need the plan (they would only wait for the same
// code to arrive).
template <bool BF16, bool SPLIT, class Start>
__device__ __forceinline__ void many_stretch(const AttnParams& p, const PartSet& part, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                             const PlanScratch& plan, uint8_t* smem, Start&& start) {
  uint8_t* ring = smem + 2 * kTileBytes;
  ManySmem& sh = *reinterpret_cast<ManySmem*>(ring + kRing * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned* const err = p.c.error;
  if (tid == 0) {
    for (int i = 0; i < kFull; ++i) mbar_init(&sh.kv_full[i], 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.kv_empty[i], 2);  // both halves, or one of them twice
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.meta_full[i], 1);
      mbar_init(&sh.meta_empty[i], 10);  // eight softmax warps, two product warps
      mbar_init(&sh.drain[i], 1);
      mbar_init(&sh.token[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i][0], 4);
      mbar_init(&sh.p_full[i][1], 4);
    }
    mbar_init(&sh.q_full, 8);
    mbar_init(&sh.unit_done, 2);
    mbar_init(&sh.join, 8);
    mbar_arrive(&sh.token[0]);  // half 0 has the first turn
    sh.failed = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp >= 8) start();
  auto failed = [&] { return *(volatile int*)&sh.failed != 0; };

  if (warp == 8) {
    // ---- loads
    unsigned bad = 0;
    int item = 0, units = 0;  // ring items (a K or a V tile each) and units so far
    auto publish = [&](const UnitMeta& u) -> bool {
      const int mi = units & 1;
      if (units >= 2) wait_or_fail(&sh.meta_empty[mi], ((units >> 1) - 1) & 1, &sh.failed, err);
      if (__any_sync(0xffffffffu, failed())) return false;
      if (lane == 0) {
        sh.meta[mi] = u;
        mbar_arrive(&sh.meta_full[mi]);
      }
      ++units;
      return true;
    };
    bool ok = true;
    plan_walk<kManyRows, SPLIT>(p, part, &plan, [&](const UnitMeta& u) -> bool {
      // the unit's queries are on their way to L2 while the unit before it is worked on
      for (int r = lane; r < u.rows; r += 32) {
        const uint16_t* q = row_query(p, u, r);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
      }
      if (!(ok = publish(u))) return false;
      auto lookup = [&](int k) {
        const int place = u.key0 + k * kKeyTile + lane * p.c.page;
        return k < u.n && lane * p.c.page < kKeyTile && place < u.key_end ? page_of(p, u.seq, place, &bad) : -1;
      };
      int next = lookup(0);
      for (int k = 0; k < u.n; ++k) {
        const int page = next;
        next = lookup(k + 1);  // in flight while this tile waits for room
        const int bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * p.c.page * kHeadDim * 2;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++item) {
          const int st = item % kRing;
          if (item >= kRing) wait_or_fail(&sh.kv_empty[st], (item / kRing - 1) & 1, &sh.failed, err);
          if (__any_sync(0xffffffffu, failed())) return ok = false;
          if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[item % kFull], bytes);
          __syncwarp();
          if (page >= 0) {
            const uint32_t dst = smem_addr(ring + st * kTileBytes) + lane * p.c.page * 128;
            tma_page(dst, kv ? &vmap : &kmap, &sh.kv_full[item % kFull], 0, u.kh, page);
            tma_page(dst + kPanelBytes, kv ? &vmap : &kmap, &sh.kv_full[item % kFull], 64, u.kh, page);
          }
        }
      }
      return true;
    });
    if (ok) {
      UnitMeta end = {};
      publish(end);
    }
    if (bad) atomicOr(err, bad);
    // no copy is in flight when the block ends, also where the others gave up
    for (int i = max(item - kRing, 0); i < item; ++i)
      if (!mbar_wait_bounded(&sh.kv_full[i % kFull], (i / kFull) & 1)) break;
  } else if (warp >= 9) {
    // ---- products of half s
    const int s = warp - 9;
    const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);
    constexpr uint32_t idesc_s = instr_desc<BF16>(false), idesc_o = instr_desc<BF16>(true);
    // Waits on several barriers at once, one a lane: a wait costs about 150 clocks even when there is nothing to wait
    // for.  All lanes see the same outcome, so the control flow is uniform.
    auto wait_all = [&](int count, uint64_t* bar, uint32_t parity) {  // lanes 0 .. count - 1, each its own bar
      bool done = lane >= count || mbar_test_wait(bar, parity);
      for (uint32_t i = 0; !__all_sync(0xffffffffu, done); ++i) {
        if (!done) done = i < 64 ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);  // it is usually near
        if ((i & 255) == 255 && __any_sync(0xffffffffu, failed() || i > kSpinLimit)) {
          if (lane == 0 && !failed()) {
            *(volatile int*)&sh.failed = 1;
            atomicOr(err, PALU_DEVERR_TIMEOUT);
          }
          return false;
        }
      }
      return true;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(1, bar, parity); };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    int tile0 = 0;            // tiles of earlier units
    uint32_t pc = 0, turns = 0;  // tiles of weights taken; turns had
    for (int unit = 0;; ++unit) {
      if (!wait(&sh.meta_full[unit & 1], (unit >> 1) & 1)) break;
      const int n = sh.meta[unit & 1].n;
      const bool both = sh.meta[unit & 1].rows > kHalf;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meta_empty[unit & 1]);
      if (n == 0 || !wait(&sh.q_full, unit & 1)) break;
      tc_fence_after();
      const uint32_t qa = q_addr + (both ? s : 0) * kTileBytes;
      auto scores = [&](int tile) {  // S = Q K^T, the keys of a tile
        const uint64_t da = smem_desc(qa, 16, 1024), db = smem_desc(ring_addr + (2 * tile % kRing) * kTileBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * kPanelBytes + (k & 3) * 32) >> 4;
          tc_mma_ss(tmem + s * 128, da + off, db + off, idesc_s, k > 0);
        }
        tc_commit(&sh.s_full[s]);
      };
      auto values = [&](int u, int tile, bool acc) {  // O += P_u V, 64 keys of a tile
        const uint64_t db = smem_desc(ring_addr + ((2 * tile + 1) % kRing) * kTileBytes + u * 8192, kPanelBytes, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_ts(tmem + 256 + s * 128, tmem + s * 128 + u * 32 + k * 8, db + (k * 2048 >> 4), idesc_o, acc || k > 0);
      };
      auto release = [&](int it) {  // the half's arrival, or both where a tile is one half's alone
        tc_commit(&sh.kv_empty[it % kRing]);
        if (!both) tc_commit(&sh.kv_empty[it % kRing]);
      };
      const int step = both ? 1 : 2, j0 = both ? 0 : s;
      bool ok = true;
      if (j0 < n) {
        const int it = 2 * (tile0 + j0);
        if (!wait(&sh.kv_full[it % kFull], (it / kFull) & 1)) break;
        if (elect_one()) {
          scores(tile0 + j0);
          release(it);
        }
        __syncwarp();
      }
      for (int j = j0; j < n; j += step) {
        const int t = tile0 + j, vi = 2 * t + 1, ki = 2 * (t + step);
        const bool more = j + step < n;
        ok = wait_all(2, lane ? &sh.kv_full[vi % kFull] : &sh.p_full[s][0], lane ? (vi / kFull) & 1 : pc & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) values(0, t, j >= step);
        __syncwarp();
        // The halves take turns with their last values and next scores: left to themselves they fall into step, both in
        // the softmax and then both waiting for the tensor cores (3,900 clocks a tile pair).
        ok = wait_all(!more ? 1 : both ? 3 : 2,
                      lane == 0   ? &sh.p_full[s][1]
                      : lane == 1 ? &sh.kv_full[ki % kFull]
                                  : &sh.token[s],
                      lane == 0 ? pc & 1 : lane == 1 ? (ki / kFull) & 1 : turns & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(1, t, true);
          if (more) {
            scores(t + step);
            if (both) mbar_arrive(&sh.token[1 - s]);
            release(vi);
            release(ki);
          } else {
            release(vi);
          }
        }
        __syncwarp();
        ++pc;
        if (more && both) ++turns;
      }
      if (!ok) break;
      commit(&sh.unit_done);
      tile0 += n;
    }
    // every product has ended before TMEM is given back
    commit(&sh.drain[s]);
    mbar_wait_bounded(&sh.drain[s], 0);
  } else {
    // ---- softmax: half `s`, a row a thread
    const int s = warp >> 2, t = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of TMEM
    const uint32_t s_addr = tmem + lanes + s * 128, o_addr = tmem + lanes + 256 + s * 128;
    int tile0 = 0;
    uint32_t sc = 0, joins = 0;
    auto join = [&] {  // the eight softmax warps meet
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.join);
      wait_or_fail(&sh.join, joins & 1, &sh.failed, err);
      ++joins;
      __syncwarp();
    };
    for (int unit = 0;; ++unit) {
      wait_or_fail(&sh.meta_full[unit & 1], (unit >> 1) & 1, &sh.failed, err);
      __syncwarp();
      if (__any_sync(0xffffffffu, failed())) break;
      const UnitMeta& m = sh.meta[unit & 1];
      if (m.n == 0) break;
      const bool both = m.rows > kHalf;
      // Q: a half's 128 rows, or each 64 of the one half's; rows behind the unit's are zeros
      {
        UnitMeta u;  // in registers: the copies' asm would have each iteration read shared memory again
        u.tok = m.tok, u.g0 = m.g0, u.kh = m.kh, u.rows = m.rows;
        const int r_base = both ? s * kHalf : 0, q_rows = both ? kHalf : kHalf / 2, q0 = both ? 0 : s * (kHalf / 2);
        const uint32_t q_tile = smem_addr(smem) + (both ? s : 0) * kTileBytes;
        for (int i = t; i < q_rows * 16; i += kHalf) {
          const int r = q0 + (i >> 4), ch = i & 15;
          const bool there = r_base + r < u.rows;
          const uint16_t* src = there ? row_query(p, u, r_base + r) + ch * 8 : p.q;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(panel_addr(q_tile, r, ch)), "l"(src),
                       "r"(there ? 16 : 0)
                       : "memory");
        }
        cp_async_commit();
        cp_async_wait<0>();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
      }
      const int r = (both ? s * kHalf : 0) + t;  // row of the unit
      const bool live = r < m.rows;
      const int lim = live ? unit_row_limit(p, plan, m, r) : 0x7fffffff;
      float ref = 0.f, l = 0.f;  // the weights' reference (log2), their sum
      bool seen = false;         // whether there is a reference yet
      const int step = both ? 1 : 2;
      for (int j = both ? 0 : s; j < m.n; j += step, ++sc) {
        const int tile_key = m.key0 + j * kKeyTile, valid = m.key_end - tile_key;
        if (valid < kKeyTile) {
          // the last tile's values behind the last key: 0 * NaN is NaN, so they are zeroed before the product (by both
          // halves, where both use them)
          const int vi = 2 * (tile0 + j) + 1;
          wait_or_fail(&sh.kv_full[vi % kFull], (vi / kFull) & 1, &sh.failed, err);
          const uint32_t v_tile = smem_addr(ring + (vi % kRing) * kTileBytes);
          for (int i = t; i < (kKeyTile - valid) * 16; i += kHalf)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(panel_addr(v_tile, valid + (i >> 4), i & 15)), "r"(0)
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        wait_or_fail(&sh.s_full[s], sc & 1, &sh.failed, err);
        __syncwarp();
        tc_fence_after();
        // The scores pass twice, 64 at a time, for the maximum and for the weights (a thread with all 128 spills).  Both
        // loops are kept rolled: a launch has to fetch its code, and the softmax has time to spare.
        uint32_t x[64];
        float* const f = reinterpret_cast<float*>(x);
        const int seen_here = lim - tile_key;
        const bool cut = __any_sync(0xffffffffu, seen_here < kKeyTile);
        auto load = [&](int u) {
          tc_ld32(x, s_addr + 64 * u);
          tc_ld32(x + 32, s_addr + 64 * u + 32);
          tc_wait_ld(x);
          tc_wait_ld(x + 32);
          if (cut) {
            const int n = seen_here - 64 * u;
#pragma unroll
            for (int i = 0; i < 64; ++i) f[i] = i < n ? f[i] : -INFINITY;
          }
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          load(u);
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], f[i + q], f[i + 4 + q]);
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * p.scale_log2;
        // raise the maximum?  O of this half is complete up to the tile before: its product was issued before these scores
        float alpha = 1.f;
        constexpr float kLift = BF16 ? 0.f : 6.f;
        if (top > ref + (kLift + kRaise) || (!seen && top != -INFINITY)) {
          alpha = seen ? ex2f_(ref - (top - kLift)) : 1.f;  // nothing but zeros so far: no factor
          ref = top - kLift;
          seen = true;
          l *= alpha;
        }
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            uint32_t o[16];
            tc_ld16(o, o_addr + 16 * i);
            tc_wait_ld16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tc_st16(o_addr + 16 * i, o);
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          load(u);
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a = f[2 * i], b = f[2 * i + 1];
            fma2(a, b, p.scale_log2, -ref);
            a = ex2f_(a);
            b = ex2f_(b);
            add2(sum[2 * (i & 1)], sum[2 * (i & 1) + 1], a, b);
            w[i] = pack2<BF16>(a, b);
          }
          tc_st32(s_addr + 32 * u, w);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[s][u]);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // ---- the unit's result
      wait_or_fail(&sh.unit_done, unit & 1, &sh.failed, err);
      __syncwarp();
      tc_fence_after();
      if (__any_sync(0xffffffffu, failed())) break;
      // A unit of up to 128 rows has an accumulator of even and one of odd tiles (if it had more than one), in the
      // same lanes of TMEM; the halves exchange their maxima and sums and each takes 64 columns of the joined rows.
      // Of a larger unit each half has its own rows.  A warp turns 128 bytes of its 32 rows around in shared memory
      // (Q is free), so that it stores whole lines.
      if (!seen) ref = -INFINITY;
      float2(*const ml)[kHalf] = reinterpret_cast<float2(*)[kHalf]>(smem + 8 * kStageBytes);  // behind the staging areas
      float fa = 1.f, fb = 0.f;
      if (!both) {
        ml[s][t] = make_float2(ref, l);
        join();
        if (m.n > 1) {
          const float2 o0 = ml[0][t], o1 = ml[1][t];
          ref = fmaxf(o0.x, o1.x);
          const float z = ref == -INFINITY ? 0.f : ref;
          fa = ex2f_(o0.x - z);
          fb = ex2f_(o1.x - z);
          l = o0.y * fa + o1.y * fb;
        } else {
          ref = ml[0][t].x;
          l = ml[0][t].y;
        }
      }
      const uint32_t o0_addr = tmem + lanes + 256 + (both ? s * 128 : 0);
      const int dest = m.dest;
      const long long set = dest == kToRow ? (m.prefix ? 0 : (long long)p.N * p.Hq) : 0;
      if (dest != kToOut && live && (both || s == 0)) {
        float2* to = dest == kToRow ? p.row_ml + set + row_index(p, m, r) : part.ml + (long long)dest * kManyRows + r;
        *to = make_float2(ref, l);
      }
      const float inv = dest != kToOut ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
      fa *= inv;
      fb *= inv;
      float* const stage = reinterpret_cast<float*>(smem + warp * kStageBytes);
      const int r_warp = (both ? s * kHalf : 0) + 32 * (warp & 3);  // first of the warp's rows
      UnitMeta u;
      u.tok = m.tok, u.g0 = m.g0, u.kh = m.kh, u.rows = m.rows;
      const bool two = !both && m.n > 1;
      auto columns = [&](int c, uint32_t* o) {  // 32 of O, joined and scaled
        float* v = reinterpret_cast<float*>(o);
        tc_ld32(o, o0_addr + c);
        tc_wait_ld(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= fa;
        if (two) {
          uint32_t y[32];
          tc_ld32(y, o0_addr + 128 + c);
          tc_wait_ld(y);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = fmaf(__uint_as_float(y[k]), fb, v[k]);
        }
      };
      const int c0 = both ? 0 : 64 * s, c1 = both ? 128 : 64 * s + 64;
      if (dest == kToOut) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 64) {
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            columns(c + 32 * h, o);
            const float* v = reinterpret_cast<const float*>(o);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(stage + lane * 36 + 16 * h + 4 * k) =
                  make_uint4(pack2<BF16>(v[8 * k], v[8 * k + 1]), pack2<BF16>(v[8 * k + 2], v[8 * k + 3]),
                             pack2<BF16>(v[8 * k + 4], v[8 * k + 5]), pack2<BF16>(v[8 * k + 6], v[8 * k + 7]));
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 8 lanes a row
            const int rr = 4 * k + (lane >> 3);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + rr * 36 + 4 * (lane & 7));
            if (r_warp + rr < u.rows)
              *reinterpret_cast<uint4*>(p.out + row_index(p, u, r_warp + rr) * kHeadDim + c + 8 * (lane & 7)) = x;
          }
        }
      } else {
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32];
          columns(c, o);
          const float* v = reinterpret_cast<const float*>(o);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4*>(stage + lane * 36 + 4 * k) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 8 lanes a row
            const int rr = 4 * k + (lane >> 3);
            const float4 x = *reinterpret_cast<const float4*>(stage + rr * 36 + 4 * (lane & 7));
            if (r_warp + rr < u.rows) {
              float* acc = dest == kToRow ? p.row_acc + (set + row_index(p, u, r_warp + rr)) * kHeadDim
                                          : part.acc + ((long long)dest * kManyRows + r_warp + rr) * kHeadDim;
              *reinterpret_cast<float4*>(acc + c + 4 * (lane & 7)) = x;
            }
          }
        }
      }
      join();  // the staging areas have been read: Q may be written again
      tc_fence_before();
      tile0 += m.n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meta_empty[unit & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tc_dealloc(tmem);
}

}  // namespace palu
