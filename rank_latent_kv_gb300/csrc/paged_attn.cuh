// The work plan of the paged attention, shared by its kernels.
//
// softmax(q K^T) V splits over the keys: a part of them gives, per row, its
// maximum m, its sum l of 2^(s - m) and its weighted sum of values; parts are
// joined by rescaling to the common maximum.  So the keys that the batch
// shares and a sequence's own are two parts, and each is cut further where
// there are fewer rows than SMs.
//
// A row is one (new token, query head).  The rows that attend to the same
// keys through the same KV head form units of up to R rows, R the row tile of
// the kernel that takes them:
//   prefix units (KV head, row tile): all rows of the batch, keys [0, S0);
//   own units (sequence, row tile, KV head): keys [S0, the last row's place].
// Units in this order, each as many 128-key tiles long as its keys are, make
// one line of tiles; CTA c of a persistent grid takes tiles [c W, (c+1) W) of
// it, so every SM has the same number of tiles whatever the lengths.  A CTA's
// stretch begins with at most one unit that an earlier CTA began and ends with
// at most one that a later CTA ends: two partial results a CTA at most.
// Units inside are complete: they go straight to the output, or, where the
// prefix and the own keys have still to be joined, to one record a row each.
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace palu {

constexpr int kKeyTile = 128;
constexpr int kTileBytes = kKeyTile * kHeadDim * 2;  // 32 KB of keys or values
constexpr int kPanelBytes = kTileBytes / 2;          // 64 of the 128 channels, rows of 128 swizzled bytes

// Partial results of one kernel launch: 2 slots a CTA, each R rows.
struct PartSet {
  float2* ml;      // [2 grid][R] (m, l)
  float* acc;      // [2 grid][R][128]
  long long* plan; // [0]: W; [1 + b]: first tile of sequence b's own units
  int grid, R;
};

struct AttnParams {
  PagedView c;
  const uint16_t* q;
  long long qs0, qs1;
  const int* offsets;
  uint16_t* out;
  float2* row_ml;   // [2][N Hq]: complete prefix units, complete own units (where there is a prefix)
  float* row_acc;   // [2][N Hq][128]
  PartSet part;
  int N, max_new, Hq, Gq;
  int S0;           // shared tokens
  int do_prefix, do_own;
  float scale_log2;
};

// A sequence's rows and length; n = 0 for one whose offsets make no sense.
struct SeqSpan {
  int tok0, n, len;
};

__device__ __forceinline__ SeqSpan seq_span(const AttnParams& p, int b, unsigned* bad) {
  const int o0 = __ldg(p.offsets + b), o1 = __ldg(p.offsets + b + 1);
  const long long len = __ldg(p.c.lengths + b), cap = (long long)p.c.width * p.c.page;
  SeqSpan s;
  s.tok0 = o0;
  s.n = (o0 >= 0 && o1 >= o0 && o1 <= p.N && (long long)o1 - o0 <= p.max_new) ? o1 - o0 : 0;
  if (s.n == 0 && o1 != o0) *bad |= PALU_DEVERR_SPAN;
  if (len > cap) *bad |= PALU_DEVERR_CAPACITY;
  s.len = (int)(len < 0 ? 0 : len > cap ? cap : len);
  return s;
}

// Tokens that row r (token r / Gq of the sequence) sees: may be <= 0.
__device__ __forceinline__ int row_limit(const SeqSpan& s, int token) { return s.len - s.n + token + 1; }

// 128-key tiles of own units in row tile rt.
template <int R>
__device__ __forceinline__ int own_tiles(const SeqSpan& s, int rt, int Gq, int S0) {
  const int last = min((rt + 1) * R, s.n * Gq) - 1;
  const int keys = row_limit(s, last / Gq) - S0;
  return keys > 0 ? (keys + kKeyTile - 1) / kKeyTile : 0;
}

// Tiles of all own units of a sequence.
template <int R>
__device__ __forceinline__ long long seq_tiles(const SeqSpan& s, int Gq, int S0, int kv_heads) {
  long long t = 0;
  for (int rt = 0; rt * R < s.n * Gq; ++rt) t += own_tiles<R>(s, rt, Gq, S0);
  return t * kv_heads;
}

__host__ __device__ inline long long prefix_tiles_of(int S0) { return (S0 + kKeyTile - 1) / kKeyTile; }

// Where a finished unit goes.
enum { kToOut = -1, kToRow = -2 };

// A CTA's stretch of a unit: `n` tiles from key0 on, as the loading warp hands
// it to the others.
struct UnitMeta {
  int key0;     // place of the first key
  int key_end;  // behind the unit's last key (inside the stretch's last tile, or behind it)
  int n;        // tiles; 0: the line has ended
  int kh;       // KV head
  int row0;     // first row of the row tile, among the unit set's rows
  int rows;     // rows in it
  int tok0;     // token of row 0 of the set
  int base;     // own units: the place of the set's first new token
  int seq;      // row of the page table
  int prefix;   // a prefix unit: each row's own limit is looked up
  int dest;     // slot, kToOut or kToRow
};

// The CTA's stretch of the line, found by the whole CTA (blockDim.x threads).
struct PlanScratch {
  long long warp_sum[16];
  long long w0, w1, base;
  int b;
};

template <int R>
__device__ __forceinline__ void plan_start(const AttnParams& p, PlanScratch* sc) {
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, nwarp = nthr >> 5;
  const int B = p.c.batch, Hkv = p.c.kv_heads;
  const long long units0 = p.do_prefix ? (long long)Hkv * (((long long)p.N * p.Gq + R - 1) / R) : 0;
  const long long prefix = units0 * prefix_tiles_of(p.S0);
  const int per = (B + nthr - 1) / nthr;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  unsigned bad = 0;
  long long mine = 0;
  if (p.do_own)
    for (int b = b0; b < b1; ++b) mine += seq_tiles<R>(seq_span(p, b, &bad), p.Gq, p.S0, Hkv);
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) sc->warp_sum[warp] = incl;
  if (tid == 0) sc->b = -1;
  __syncthreads();
  long long before = prefix, total = prefix;
  for (int w = 0; w < nwarp; ++w) {
    if (w < warp) before += sc->warp_sum[w];
    total += sc->warp_sum[w];
  }
  before += incl - mine;
  const long long W = max((total + gridDim.x - 1) / gridDim.x, 1LL);
  const long long w0 = (long long)blockIdx.x * W, w1 = min(w0 + W, total);
  if (p.do_own) {
    // the thread whose sequences hold the CTA's first own tile walks them; CTA 0 writes the plan down
    const long long at = max(w0, prefix);
    const bool here = at < w1 && at >= before && at < before + mine;
    if (here || blockIdx.x == 0) {
      long long base = before;
      for (int b = b0; b < b1; ++b) {
        if (blockIdx.x == 0) p.part.plan[1 + b] = base;
        const long long t = seq_tiles<R>(seq_span(p, b, &bad), p.Gq, p.S0, Hkv);
        if (here && at >= base && at < base + t) {
          sc->b = b;
          sc->base = base;
        }
        base += t;
      }
    }
    if (blockIdx.x == 0 && bad) atomicOr(p.c.error, bad);
  }
  if (tid == 0) {
    sc->w0 = w0;
    sc->w1 = w1;
    if (blockIdx.x == 0) p.part.plan[0] = W;
  }
  __syncthreads();
}

// Calls unit(meta) for each unit that the CTA's stretch of the line touches, in
// order, until it returns false: run by one warp, all its lanes.
template <int R, class F>
__device__ __forceinline__ void plan_walk(const AttnParams& p, const PlanScratch* sc, F&& unit) {
  const int Hkv = p.c.kv_heads;
  const long long w1 = sc->w1;
  long long pos = sc->w0;
  const int tiles0 = (int)prefix_tiles_of(p.S0);
  const int all_rows = p.N * p.Gq;
  const int rts = (all_rows + R - 1) / R;
  const long long prefix = p.do_prefix ? (long long)Hkv * rts * tiles0 : 0;
  const int cta = blockIdx.x;
  UnitMeta m;
  // the unit [u0, u0 + n) and the stretch of it that starts at pos
  auto run_unit = [&](long long u0, int n, int key_base, int key_end) -> bool {
    const int k0 = (int)(pos - u0);
    const int k1 = (int)min((long long)n, k0 + (w1 - pos));
    m.dest = k0 > 0 ? 2 * cta : k1 < n ? 2 * cta + 1 : p.S0 > 0 ? kToRow : kToOut;
    m.key0 = key_base + k0 * kKeyTile;
    m.key_end = key_end;
    m.n = k1 - k0;
    pos += m.n;
    return unit(m);
  };
  while (pos < w1 && pos < prefix) {
    const int u = (int)(pos / tiles0);
    m.kh = u / rts;
    const int rt = u - m.kh * rts;
    m.row0 = rt * R;
    m.rows = min(R, all_rows - m.row0);
    m.tok0 = m.base = m.seq = 0;
    m.prefix = 1;
    if (!run_unit((long long)u * tiles0, tiles0, 0, p.S0)) return;
  }
  if (!p.do_own || pos >= w1) return;
  long long base = sc->base;
  unsigned bad = 0;
  for (int b = sc->b; b >= 0 && b < p.c.batch && pos < w1; ++b) {
    const SeqSpan s = seq_span(p, b, &bad);
    m.tok0 = s.tok0;
    m.base = s.len - s.n;
    m.seq = b;
    m.prefix = 0;
    for (int rt = 0; rt * R < s.n * p.Gq; ++rt) {
      const int n = own_tiles<R>(s, rt, p.Gq, p.S0);
      if (!n) continue;
      if (pos >= base + (long long)n * Hkv) {
        base += (long long)n * Hkv;
        continue;
      }
      m.row0 = rt * R;
      m.rows = min(R, s.n * p.Gq - m.row0);
      const int end = row_limit(s, (m.row0 + m.rows - 1) / p.Gq);
      for (m.kh = (int)((pos - base) / n); m.kh < Hkv && pos < w1; ++m.kh)
        if (!run_unit(base + (long long)m.kh * n, n, p.S0, end)) return;
      base += (long long)n * Hkv;
      if (pos >= w1) return;
    }
  }
}

// The limit of a row of the unit: how many of the sequence's tokens it sees.
__device__ __forceinline__ int unit_row_limit(const AttnParams& p, const UnitMeta& m, int r) {
  const int tok = (m.row0 + r) / p.Gq;
  if (!m.prefix) return m.base + tok + 1;
  // token numbers of the whole call: the row's sequence
  int lo = 0, hi = p.c.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.offsets + mid) <= tok)
      lo = mid;
    else
      hi = mid;
  }
  unsigned bad = 0;
  const SeqSpan s = seq_span(p, lo, &bad);
  const int i = tok - s.tok0;
  return i >= 0 && i < s.n ? min(row_limit(s, i), p.S0) : 0;
}

// The page that holds token `place` of table row `seq` (0 and an error bit for
// an id outside the pool).
__device__ __forceinline__ int page_of(const AttnParams& p, int seq, int place, unsigned* bad) {
  const int page = __ldg(p.c.table + (long long)seq * p.c.width + (place >> p.c.page_shift));
  if (page >= 0 && page < p.c.n_pages) return page;
  *bad |= PALU_DEVERR_PAGE;
  return 0;
}

// One page of one head, 64 channels from x on, into a panel.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(0), "r"(head), "r"(page)
      : "memory");
}

// Shared-memory address of 16-byte chunk ch (0..15) of a tile's row, in the
// 128-byte swizzle the copies write.
__device__ __forceinline__ uint32_t panel_addr(uint32_t tile, int row, int ch) {
  return tile + (ch >> 3) * kPanelBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// A wait that gives up sets the error word, and `failed` for the block: every
// role then runs on to its end without waiting (what it computes is void).
__device__ __forceinline__ void wait_or_fail(uint64_t* bar, uint32_t parity, int* failed, unsigned* error) {
  if (*(volatile int*)failed) return;
  if (!mbar_wait_bounded(bar, parity)) {
    *(volatile int*)failed = 1;
    atomicOr(error, PALU_DEVERR_TIMEOUT);
  }
}

// A launch; `dependent`: it may begin while the one before it on the stream still
// runs, and waits for it inside.
template <class K, class... Args>
palu_status launch(K kernel, int grid, int threads, int smem, bool dependent, cudaStream_t stream, const char* what,
                          Args... args) {
  int per_sm = 0;
  palu_status st = kernel_occupancy(reinterpret_cast<const void*>(kernel), threads, smem, &per_sm);
  if (st != PALU_OK) return st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, args...), what);
}

// The kernel for many rows (paged_many.cu).
constexpr int kManyRows = 256;
palu_status launch_many(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream);

}  // namespace palu
