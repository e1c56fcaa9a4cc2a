// The pass that normalises and rotates queries and keys, for the kernels that
// do it on the way somewhere: into head-major tensors and fp16 or bf16 pages
// (paged_append.cu), into pages of 4-bit codes (paged4_append.cu).
#pragma once

#include "paged.cuh"

namespace palu {

constexpr int kRunHeads = 4;       // heads a half-warp takes
constexpr int kAppendThreads = 256;

struct QkParams {
  palu_qk_transform tr;
  const uint16_t *q, *k, *v;
  long long qs0, qs1, qs2, ks0, ks1, ks2, vs1, vs2;  // batch, token, head strides in elements
  const long long* positions;
  uint16_t *q_out, *k_out;
  unsigned int* error;
  long long rows;      // tokens of all sequences
  long long tokens;    // tokens of a sequence (dense form)
  int hq, hk, q_runs, k_runs, runs;
  const int* offsets;  // paged form
  PagedView c;
};

// A row's two pieces of four channels a lane: the norm (by w, where there is
// one), then the rotation of the lane's four pairs: (x0, x4) .. (x3, x7), or
// (x0, x1) .. (x6, x7) when interleaved.
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void transform_row(uint2& lo, uint2& hi, bool norm, const float (&w)[8], bool turn,
                                              const float4& co, const float4& si, float eps, unsigned mask) {
  float x[8];
  const uint32_t raw[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(raw[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  if (norm) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
    for (int m = 8; m; m >>= 1) s += __shfl_xor_sync(mask, s, m);
    const float r = rsqrtf(s * (1.f / kHeadDim) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (turn) {
    const float c[4] = {co.x, co.y, co.z, co.w}, s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = INTERLEAVED ? 2 * i : i, k = INTERLEAVED ? 2 * i + 1 : i + 4;
      const float a = x[j], b = x[k];
      x[j] = a * c[i] - b * s[i];
      x[k] = b * c[i] + a * s[i];
    }
  }
  lo = make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
  hi = make_uint2(pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}

// Rows 16 tile .. 16 tile + 15 of a run of heads, by a CTA's half-warps.
template <bool BF16, bool INTERLEAVED, bool PAGED>
__device__ __forceinline__ void transform_tile(const QkParams& p, int tile, int run) {
  const int lane = threadIdx.x & 15;
  const unsigned mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  const long long row = (long long)tile * (kAppendThreads / 16) + (threadIdx.x >> 4);
  if (row >= p.rows) return;
  // which heads: queries, keys, then (paged form) values
  const int kind = run < p.q_runs ? 0 : run < p.q_runs + p.k_runs ? 1 : 2;
  const int h0 = (kind == 0 ? run : kind == 1 ? run - p.q_runs : run - p.q_runs - p.k_runs) * kRunHeads;
  const int nh = min(kRunHeads, (kind == 0 ? p.hq : p.hk) - h0);
  const long long bi = PAGED ? 0 : row / p.tokens, ti = PAGED ? row : row - bi * p.tokens;
  const uint16_t* src = kind == 0   ? p.q + bi * p.qs0 + ti * p.qs1 + (long long)h0 * p.qs2
                        : kind == 1 ? p.k + bi * p.ks0 + ti * p.ks1 + (long long)h0 * p.ks2
                                    : p.v + ti * p.vs1 + (long long)h0 * p.vs2;
  const long long hs = kind == 0 ? p.qs2 : kind == 1 ? p.ks2 : p.vs2;
  // the lane's channels: ca .. ca+3 and cb .. cb+3
  const bool pairs = lane < (p.tr.rope_dim >> 3);
  const int ca = !INTERLEAVED && pairs ? 4 * lane : 8 * lane;
  const int cb = !INTERLEAVED && pairs ? (p.tr.rope_dim >> 1) + 4 * lane : 8 * lane + 4;
  uint2 lo[kRunHeads], hi[kRunHeads];
#pragma unroll
  for (int i = 0; i < kRunHeads; ++i)
    if (i < nh) {
      lo[i] = __ldg(reinterpret_cast<const uint2*>(src + i * hs + ca));
      hi[i] = __ldg(reinterpret_cast<const uint2*>(src + i * hs + cb));
    }

  // the token's place, and whether it may be written
  long long pos = 0, page = 0;
  int slot = 0;
  unsigned bad = 0;
  if (PAGED) {
    const int b = find_sequence(p.offsets, p.c.batch, (int)row, lane, mask);
    const int o0 = __ldg(p.offsets + b), o1 = __ldg(p.offsets + b + 1);
    if (row >= __ldg(p.offsets + p.c.batch)) return;  // behind the last sequence
    const long long len = __ldg(p.c.lengths + b);
    if (o0 < 0 || row < o0 || row >= o1 || o1 > p.rows || len < o1 - o0)
      bad = PALU_DEVERR_SPAN;
    else if (len > (long long)p.c.width * p.c.page)
      bad = PALU_DEVERR_CAPACITY;
    else {
      pos = len - o1 + row;
      slot = (int)(pos & (p.c.page - 1));
      page = __ldg(p.c.table + (long long)b * p.c.width + (pos >> p.c.page_shift));
      if (page < 0 || page >= p.c.n_pages) bad = PALU_DEVERR_PAGE;
    }
  }
  const bool turn = kind < 2 && pairs;
  float4 co = {}, si = {};
  if (p.tr.cos_sin != nullptr) {
    if (p.positions) pos = __ldg(p.positions + row);
    if (!bad && (pos < 0 || pos >= p.tr.n_positions)) bad = PALU_DEVERR_POSITION;
    if (!bad && turn) {
      const float* cs = p.tr.cos_sin + pos * p.tr.rope_dim + 4 * lane;
      co = __ldg(reinterpret_cast<const float4*>(cs));
      si = __ldg(reinterpret_cast<const float4*>(cs + (p.tr.rope_dim >> 1)));
    }
  }
  if (bad && lane == 0 && p.error) atomicOr(p.error, bad);
  if (bad && PAGED && kind > 0) return;  // nothing of it is appended

  const uint16_t* wsrc = static_cast<const uint16_t*>(kind == 0 ? p.tr.q_weight : kind == 1 ? p.tr.k_weight : nullptr);
  float w[8] = {};
  if (wsrc) {
    const uint2 wl = __ldg(reinterpret_cast<const uint2*>(wsrc + ca)), wh = __ldg(reinterpret_cast<const uint2*>(wsrc + cb));
    const uint32_t raw[4] = {wl.x, wl.y, wh.x, wh.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(raw[i]);
      w[2 * i] = f.x;
      w[2 * i + 1] = f.y;
    }
  }
  uint16_t* dst;
  long long ds;  // between heads
  if (PAGED) {
    if (kind == 0) {
      dst = p.q_out + (row * p.hq + h0) * kHeadDim;
      ds = kHeadDim;
    } else if (kind == 1) {
      dst = p.c.k + page * p.c.ks0 + h0 * p.c.ks1 + slot * p.c.ks2;
      ds = p.c.ks1;
    } else {
      dst = p.c.v + page * p.c.vs0 + h0 * p.c.vs1 + slot * p.c.vs2;
      ds = p.c.vs1;
    }
  } else {
    dst = (kind == 0 ? p.q_out : p.k_out) + ((bi * (kind == 0 ? p.hq : p.hk) + h0) * p.tokens + ti) * kHeadDim;
    ds = p.tokens * kHeadDim;
  }
  const uint32_t nan2 = 0x7fff7fffu;  // a NaN in either type
#pragma unroll
  for (int i = 0; i < kRunHeads; ++i) {
    if (i < nh) {  // the same for all 16 lanes
      if (bad)
        lo[i] = hi[i] = make_uint2(nan2, nan2);
      else if (kind < 2)
        transform_row<BF16, INTERLEAVED>(lo[i], hi[i], wsrc != nullptr, w, turn, co, si, p.tr.eps, mask);
      *reinterpret_cast<uint2*>(dst + i * ds + ca) = lo[i];
      *reinterpret_cast<uint2*>(dst + i * ds + cb) = hi[i];
    }
  }
}

// Host checks of the calls' operands.
palu_status transform_check(const palu_qk_transform* t);
palu_status rows_check(const char* name, const void* p, const int64_t* strides, int n);

}  // namespace palu
