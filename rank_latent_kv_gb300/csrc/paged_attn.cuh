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
//   prefix units (KV head, row tile): all rows of the batch, keys [0, S0), or
//     up to the longest length where no sequence has all of them: behind it
//     pages may hold anything, and 0 * NaN is NaN;
//   own units (sequence, row tile, KV head): keys [S0, the last row's place].
// Units in this order make one line, measured in ticks: a unit takes a fixed
// number for its beginning and end, then some for each of its 128-key tiles
// (LineCost).  CTA c of a persistent grid takes the tiles that begin in
// [c W, (c+1) W), so every SM has the same work whatever the lengths.  Where
// the prefix has many rows and the own units few, each has a line and CTAs of
// its own, divided by the two lines' lengths (split_ctas).  A CTA's
// stretch begins with at most one unit that an earlier CTA began and ends with
// at most one that a later CTA ends: two partial results a CTA at most.  Units
// inside are complete: they go straight to the output, or, where the prefix
// and the own keys have still to be joined, to one record a row each.
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace palu {

constexpr int kKeyTile = 128;
constexpr int kTileBytes = kKeyTile * kHeadDim * 2;  // 32 KB of keys or values
constexpr int kPanelBytes = kTileBytes / 2;          // 64 of the 128 channels, rows of 128 swizzled bytes

// A CTA's stretch of a unit: `n` tiles from key0 on, as the loading warp hands
// it to the others.
struct UnitMeta {
  int key0;     // place of the first key
  int key_end;  // behind the unit's last key (inside the stretch's last tile, or behind it)
  int n;        // tiles; 0: the line has ended
  int kh;       // KV head
  int rows;     // rows of the row tile
  int tok;      // token of its first row, and that row's query head in the group
  int g0;
  int pos;      // own units: the place of that token
  int seq;      // row of the page table
  int prefix;   // a prefix unit: each row's own limit is looked up
  int dest;     // slot, kToOut or kToRow
  int parts;    // CTAs that hold a part of the unit, where this is its first one
};

// Partial results of a line: 2 slots a CTA, each R rows.
struct PartSet {
  float2* ml;       // [2 grid][R] (m, l)
  float* acc;       // [2 grid][R][128]
  long long* plan;  // [0]: W; [1 + b]: where sequence b's own units begin; [1 + B]: the prefix units' last key
  UnitMeta* begun;  // [SMs]: the unit that CTA c begins and a later one ends (rows 0: none)
  int R;
};

struct AttnParams {
  PagedView c;
  const uint16_t* q;
  long long qs0, qs1;
  const int* offsets;
  uint16_t* out;
  float2* row_ml;   // [2][N Hq]: complete prefix units, complete own units (where there is a prefix)
  float* row_acc;   // [2][N Hq][128]
  PartSet part;     // the line, or the own units'
  PartSet prefix;   // the prefix units', where they have one
  int N, max_new, Hq, Gq;
  int gq_mul;       // ceil(2^16 / Gq)
  int S0;           // shared tokens
  float scale_log2;
};

// What a unit costs, in ticks of kClocks, in the kernel with row tiles of R: to
// begin and end it, and a 128-key tile of it.  FOUR: over pages of 4-bit codes.
template <int R, bool FOUR>
struct LineCost {
  static __device__ int unit(int rows) { return 2; }  // 5,700 clocks
  static __device__ int tile(int rows) { return 1; }  // 2,900
  static constexpr int kMaxTile = 1;
  static constexpr float kClocks = 2900.f;
};
// Measured: 1520 units of 256 rows and 4 tiles take
// 34,000 clocks each, of 40 rows and 1 or 4 tiles 15,000 and 22,600; in long
// units a tile of 256 rows takes 3,100 and one of up to 128 rows 2,900 (the
// time of its 64 KB at memory speed).
constexpr int kManyRows = 256;
template <>
struct LineCost<kManyRows, false> {
  static __device__ int unit(int rows) { return rows > kManyRows / 2 ? 100 : 60; }
  static __device__ int tile(int rows) { return rows > kManyRows / 2 ? 16 : 14; }
  static constexpr int kMaxTile = 16;
  static constexpr float kClocks = 200.f;
};
// Made from codes: of up to 128 rows a tile takes 2,300 clocks and a unit 17,000 more (with 60 and 14 here 77 sequences
// of 5 tokens behind up to 1,500 keys, 28 heads of 4, took 67 us instead of 63).  Equal units, 1 to 6 a CTA of 1 to 32
// tiles, fitted: 35 to 128 rows 11,000 to 15,000 clocks a unit and 3,100 a tile, 140 and 256 rows 21,000 to 26,000 and
// 5,300 (a unit as 4.0 to 4.8 tiles; 100 / 22 is 4.5).
template <>
struct LineCost<kManyRows, true> {
  static __device__ int unit(int rows) { return rows > kManyRows / 2 ? 100 : 85; }
  static __device__ int tile(int rows) { return rows > kManyRows / 2 ? 22 : 12; }
  static constexpr int kMaxTile = 22;
  static constexpr float kClocks = 200.f;
};
// A tile of codes is 20 KB.  Equal units as above: up to 8 rows 7,100 clocks a unit and 1,020 a tile, up to 16 rows
// 11,800 and 1,790 (a unit as 6.9 and 6.6 tiles).
template <int R>
struct LineCost<R, true> {
  static __device__ int unit(int rows) { return 6; }
  static __device__ int tile(int rows) { return 1; }
  static constexpr int kMaxTile = 1;
  static constexpr float kClocks = 1000.f;
};

// Row r (of a unit) -> token and query head, r < 256: g0 + r < 320 and Gq <= 64,
// for which the multiplication is exact (320 * 64 < 2^16).
__device__ __forceinline__ void row_place(const AttnParams& p, const UnitMeta& m, int r, int* tok, int* head) {
  const int x = m.g0 + r, t = (x * p.gq_mul) >> 16;
  *tok = m.tok + t;
  *head = m.kh * p.Gq + x - t * p.Gq;
}
__device__ __forceinline__ long long row_index(const AttnParams& p, const UnitMeta& m, int r) {
  int tok, head;
  row_place(p, m, r, &tok, &head);
  return (long long)tok * p.Hq + head;
}
__device__ __forceinline__ const uint16_t* row_query(const AttnParams& p, const UnitMeta& m, int r) {
  int tok, head;
  row_place(p, m, r, &tok, &head);
  return p.q + tok * p.qs0 + head * p.qs1;
}

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
  if ((s.n == 0 && o1 != o0) || (b == 0 && o0 != 0)) *bad |= PALU_DEVERR_SPAN;
  if (len > cap) *bad |= PALU_DEVERR_CAPACITY;
  s.len = (int)(len < 0 ? 0 : len > cap ? cap : len);
  return s;
}

// Tokens that row r (token r / Gq of the sequence) sees: may be <= 0.
__device__ __forceinline__ int row_limit(const SeqSpan& s, int token) { return s.len - s.n + token + 1; }

// 128-key tiles of an own unit with rows [row0, row0 + rows) of a sequence.
__device__ __forceinline__ int own_tiles(const SeqSpan& s, int row0, int rows, int Gq, int S0) {
  const int keys = row_limit(s, (row0 + rows - 1) / Gq) - S0;
  return keys > 0 ? (keys + kKeyTile - 1) / kKeyTile : 0;
}

// a / b, for quotients below 2^17 (CTAs, KV heads): a float estimate and its
// correction, where a 64-bit division is a hundred instructions to be fetched.
__device__ __forceinline__ int div_small(long long a, long long b) {
  int q = (int)__fdividef((float)a, (float)b);
  while ((long long)q * b > a) --q;
  while ((long long)(q + 1) * b <= a) ++q;
  return q;
}

// Ticks of a unit of n tiles.
template <int R, bool FOUR>
__device__ __forceinline__ long long unit_ticks(int rows, int n) {
  return n ? LineCost<R, FOUR>::unit(rows) + (long long)n * LineCost<R, FOUR>::tile(rows) : 0;
}

// Ticks of a sequence's own units before row tile `rts`.
template <int R, bool FOUR>
__device__ __forceinline__ long long seq_ticks(const SeqSpan& s, int rts, int Gq, int S0, int kv_heads) {
  long long t = 0;
  for (int rt = 0; rt < rts; ++rt) {
    const int rows = min(R, s.n * Gq - rt * R);
    t += unit_ticks<R, FOUR>(rows, own_tiles(s, rt * R, rows, Gq, S0));
  }
  return t * kv_heads;
}
template <int R, bool FOUR>
__device__ __forceinline__ long long seq_ticks(const SeqSpan& s, int Gq, int S0, int kv_heads) {
  if (s.n * Gq <= R) {  // one row tile, the usual case: its last token sees everything
    const int keys = s.n ? s.len - S0 : 0;
    return unit_ticks<R, FOUR>(s.n * Gq, keys > 0 ? (keys + kKeyTile - 1) / kKeyTile : 0) * kv_heads;
  }
  return seq_ticks<R, FOUR>(s, (s.n * Gq + R - 1) / R, Gq, S0, kv_heads);
}

// Ticks of one KV head's prefix units before row tile `rts` (all: rts row tiles).
template <int R, bool FOUR>
__device__ __forceinline__ long long prefix_ticks(int all_rows, int rts, int tiles) {
  const int full = min(rts, all_rows / R);
  long long t = full * unit_ticks<R, FOUR>(R, tiles);
  if (rts > full) t += unit_ticks<R, FOUR>(all_rows - full * R, tiles);
  return t;
}

__host__ __device__ inline int prefix_tiles_of(int keys) { return (keys + kKeyTile - 1) / kKeyTile; }

// Where a finished unit goes.
enum { kToOut = -1, kToRow = -2 };

// The CTA's stretch of its line, found by THREADS of its threads, tid 0 ..
// THREADS - 1, which meet at named barrier 3.
constexpr int kPlanWarps = 20;  // the most that plan: all of paged4_both_kernel
struct PlanScratch {
  long long warp_sum[kPlanWarps];
  long long w0, w1, W, base;
  int warp_longest[kPlanWarps];
  int cta;         // where there are two lines: its number among the CTAs of its line,
  int has_prefix;  // and whether that is the prefix units'
  int b;
  int prefix_end;  // prefix units' keys: [0, prefix_end)
  int cut_prefix;  // a sequence does not see the whole prefix with all of its new tokens
};

// CTAs of `grid` for the prefix where it has many rows and the own units few: a
// line of each, of `a` clocks of prefix and `b` of own units, so that both end
// together.  The device divides, because only it knows the lengths: a table is
// as wide as the longest sequence that a program admits (32 sequences of 777
// own tokens behind 8192, 24 heads of 8: 39 us in tables for 777 and for 131,072
// tokens; with half of the table's width as a guess 42 and 786, and 120 without
// sharing).  A prefix tile takes longer where own units keep the memory busy:
// measured over all divisions of 13 calls, from a / b = 1 / 50 to 2, its clocks
// count 0.8 + 2.3 (b / (a + b))^2 times (within 4 % of the best division, 1 % on
// average; plain shares by a and b up to 54 % off).  Every CTA finds the same
// number; each kind has one at least.
__device__ __forceinline__ int split_ctas(float a, float b, int grid) {
  const float x = __fdividef(b, a + b), k = (0.8f + 2.3f * x * x) * a;
  return a > 0.f ? min(max((int)(grid * __fdividef(k, k + b) + 0.5f), 1), grid - 1) : 1;
}

// R: row tiles of the own units; RP: of the prefix units.  RP != R: a line of
// each.
template <int R, int RP, int THREADS, bool FOUR = false>
__device__ __forceinline__ void plan_start(const AttnParams& p, PlanScratch* sc, int tid) {
  constexpr int nthr = THREADS, nwarp = THREADS / 32;
  static_assert(nwarp <= kPlanWarps, "PlanScratch has a place for each warp that plans");
  constexpr bool SPLIT = R != RP;
  const int warp = tid >> 5, lane = tid & 31;
  auto meet = [] { asm volatile("bar.sync 3, %0;" ::"n"(THREADS) : "memory"); };
  const int B = p.c.batch, Hkv = p.c.kv_heads;
  const int all_rows = p.N * p.Gq;
  const int per = (B + nthr - 1) / nthr;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  unsigned bad = 0;
  long long mine = 0;
  int longest = 0;  // of the sequences that have rows
  if (tid == 0) {
    sc->b = -1;
    sc->cut_prefix = 0;
  }
  meet();
  for (int b = b0; b < b1; ++b) {
    const SeqSpan s = seq_span(p, b, &bad);
    if (s.n && row_limit(s, 0) < p.S0) sc->cut_prefix = 1;
    if (s.n) longest = max(longest, s.len);
    mine += seq_ticks<R, FOUR>(s, p.Gq, p.S0, Hkv);
    // without a prefix nothing joins parts of every row: rows that see nothing, or that are before the first
    // sequence, are zeroed here, all CTAs sharing them
    if (p.S0 == 0) {
      const int o0 = __ldg(p.offsets + b), o1 = min(__ldg(p.offsets + b + 1), p.N);
      const int z0 = b ? max(o0, 0) : 0, z1 = s.n ? min(o1, o0 + max(s.n - s.len, 0)) : o1;
      for (long long i = (long long)z0 * p.Hq * (kHeadDim / 8) + blockIdx.x; i < (long long)z1 * p.Hq * (kHeadDim / 8);
           i += gridDim.x)
        reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (p.S0) sc->warp_longest[warp] = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) sc->warp_sum[warp] = incl;
  meet();
  long long before = 0, own = 0, prefix = 0;
#pragma unroll
  for (int w = 0; w < nwarp; ++w) {
    if (w < warp) before += sc->warp_sum[w];
    own += sc->warp_sum[w];
  }
  before += incl - mine;
  if (p.S0) {
#pragma unroll
    for (int w = 0; w < nwarp; ++w) longest = max(longest, sc->warp_longest[w]);
    longest = min(longest, p.S0);
    prefix = Hkv * prefix_ticks<RP, FOUR>(all_rows, (all_rows + RP - 1) / RP, prefix_tiles_of(longest));
  }
  int cta = blockIdx.x, grid = gridDim.x;
  bool has_prefix = p.S0 > 0, has_own = true;
  if (SPLIT) {
    const int g = split_ctas((float)prefix * LineCost<RP, FOUR>::kClocks, (float)own * LineCost<R, FOUR>::kClocks, grid);
    has_prefix = cta < g;
    has_own = !has_prefix;
    grid = has_prefix ? g : grid - g;
    cta -= has_prefix ? 0 : g;
  }
  const PartSet& part = SPLIT && has_prefix ? p.prefix : p.part;
  if (!has_prefix) prefix = 0;
  before += prefix;
  const long long total = prefix + (has_own ? own : 0);
  // a stretch is never shorter than a tile, so that every CTA between a unit's first and last holds a part of it
  const long long tile = SPLIT && has_prefix ? LineCost<RP, FOUR>::kMaxTile : LineCost<R, FOUR>::kMaxTile;
  const long long W = max((total + grid - 1) / grid, tile);
  const long long w0 = cta * W, w1 = min(w0 + W, total);
  if (has_own) {
    // the thread whose sequences hold the CTA's first own tick walks them; CTA 0 writes the plan down
    const long long at = max(w0, prefix);
    const bool here = at < w1 && at >= before && at < before + mine;
    if (here || cta == 0) {
      long long base = before;
      for (int b = b0; b < b1; ++b) {
        if (cta == 0) part.plan[1 + b] = base;
        const long long t = per == 1 ? mine : seq_ticks<R, FOUR>(seq_span(p, b, &bad), p.Gq, p.S0, Hkv);
        if (here && at >= base && at < base + t) {
          sc->b = b;
          sc->base = base;
        }
        base += t;
      }
    }
    if (cta == 0 && bad) atomicOr(p.c.error, bad);
  }
  if (tid == 0) {
    sc->w0 = w0;
    sc->w1 = w1;
    sc->W = W;
    if (SPLIT) {
      sc->cta = cta;
      sc->has_prefix = has_prefix;
    }
    if (p.S0) sc->prefix_end = longest;
    if (cta == 0) {
      part.plan[0] = W;
      if (has_prefix) part.plan[1 + B] = longest;
    }
    part.begun[cta].rows = 0;
  }
  meet();
}

// Calls unit(meta) for each unit of which the CTA's stretch of the line has
// tiles, in order, until it returns false: run by one warp, all its lanes.
// SPLIT: the line is one of two, of the prefix or of the own units.
template <int R, bool SPLIT, bool FOUR = false, class F>
__device__ __forceinline__ void plan_walk(const AttnParams& p, const PartSet& part, const PlanScratch* sc, F&& unit) {
  const int Hkv = p.c.kv_heads;
  const long long w0 = sc->w0, w1 = sc->w1;
  const int cta = SPLIT ? sc->cta : blockIdx.x;
  const bool has_prefix = SPLIT ? sc->has_prefix : p.S0 > 0;
  UnitMeta m = {};
  // the tiles of a unit [u0, u0 + ticks) that begin in [w0, w1)
  auto run_unit = [&](long long u0, int n, int key_base, int key_end) -> bool {
    const int t = LineCost<R, FOUR>::tile(m.rows);
    const long long f = u0 + LineCost<R, FOUR>::unit(m.rows);
    // tiles that begin before x
    auto before = [&](long long x) -> int {
      if (x <= f) return 0;
      if (x - f >= (long long)n * t) return n;
      return ((int)(x - f) + t - 1) / t;  // n * t < 2^28
    };
    const int k0 = before(w0), k1 = before(w1);
    if (k0 == k1) return true;
    m.dest = k0 > 0 ? 2 * cta : k1 < n ? 2 * cta + 1 : p.S0 > 0 ? kToRow : kToOut;
    m.key0 = key_base + k0 * kKeyTile;
    m.key_end = key_end;
    m.n = k1 - k0;
    if (m.dest == 2 * cta + 1) {
      m.parts = div_small(f + (long long)(n - 1) * t, sc->W) - cta + 1;
      if ((threadIdx.x & 31) == 0) part.begun[cta] = m;
    }
    return unit(m);
  };
  long long base = 0;
  if (has_prefix) {
    const int all_rows = p.N * p.Gq, rts = (all_rows + R - 1) / R, tiles = prefix_tiles_of(sc->prefix_end);
    const long long head = prefix_ticks<R, FOUR>(all_rows, rts, tiles), full = unit_ticks<R, FOUR>(R, tiles);
    m.pos = m.seq = 0;
    m.prefix = 1;
    if (w0 < head * Hkv) {
      m.kh = div_small(w0, head);
      int rt = min(div_small(w0 - m.kh * head, full), rts - 1);
      for (; m.kh < Hkv; ++m.kh, rt = 0)
        for (; rt < rts; ++rt) {
          const long long u0 = m.kh * head + rt * full;
          if (u0 >= w1) return;
          m.rows = min(R, all_rows - rt * R);
          m.tok = rt * R / p.Gq;
          m.g0 = rt * R - m.tok * p.Gq;
          if (!run_unit(u0, tiles, 0, sc->prefix_end)) return;
        }
    }
  }
  if ((SPLIT && has_prefix) || sc->b < 0) return;
  base = sc->base;
  unsigned bad = 0;
  for (int b = sc->b; b < p.c.batch; ++b) {
    const SeqSpan s = seq_span(p, b, &bad);
    m.seq = b;
    m.prefix = 0;
    for (int rt = 0; rt * R < s.n * p.Gq; ++rt) {
      m.rows = min(R, s.n * p.Gq - rt * R);
      const int n = own_tiles(s, rt * R, m.rows, p.Gq, p.S0);
      if (!n) continue;
      const long long ticks = unit_ticks<R, FOUR>(m.rows, n);
      const int end = row_limit(s, (rt * R + m.rows - 1) / p.Gq), i = rt * R / p.Gq;
      m.tok = s.tok0 + i;
      m.g0 = rt * R - i * p.Gq;
      m.pos = s.len - s.n + i;
      m.kh = w0 <= base ? 0 : w0 - base >= ticks * Hkv ? Hkv : div_small(w0 - base, ticks);
      for (; m.kh < Hkv; ++m.kh) {
        const long long u0 = base + m.kh * ticks;
        if (u0 >= w1) return;
        if (!run_unit(u0, n, p.S0, end)) return;
      }
      base += ticks * Hkv;
    }
  }
}

// The limit of a row of the unit: how many of the sequence's tokens it sees.
__device__ __forceinline__ int unit_row_limit(const AttnParams& p, const PlanScratch& sc, const UnitMeta& m, int r) {
  if (m.prefix && !sc.cut_prefix) return p.S0;
  int tok, head;
  row_place(p, m, r, &tok, &head);
  if (!m.prefix) return m.pos + (tok - m.tok) + 1;
  // the row's sequence
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
  if (mbar_try_wait(bar, parity)) return;
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (*(volatile int*)failed || mbar_try_wait(bar, parity)) return;
  }
  *(volatile int*)failed = 1;
  atomicOr(error, PALU_DEVERR_TIMEOUT);
}

// A launch; `dependent`: it may begin while the one before it on the stream still
// runs, and waits for it inside.
template <class K, class... Args>
palu_status launch(K kernel, dim3 grid, int threads, int smem, bool dependent, cudaStream_t stream, const char* what,
                          Args... args) {
  int per_sm = 0;
  palu_status st = kernel_occupancy(reinterpret_cast<const void*>(kernel), threads, smem, &per_sm);
  if (st != PALU_OK) return st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, args...), what);
}

// The kernels: few rows (paged_few.cu), many rows (paged_many.cu), and a prefix of many rows with own units of few
// (paged_both.cu).
palu_status launch_few(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream);
palu_status launch_many(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream);
palu_status launch_both(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream);
// Over pages of 4-bit codes (paged4_few.cu, paged4_many.cu, paged4_both.cu).
palu_status launch_few4(const AttnParams& p, bool bf16, cudaStream_t stream);
palu_status launch_many4(const AttnParams& p, bool bf16, cudaStream_t stream);
palu_status launch_both4(const AttnParams& p, bool bf16, cudaStream_t stream);

}  // namespace palu
