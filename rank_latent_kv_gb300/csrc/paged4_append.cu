// The 4-bit paged cache's descriptor, new tokens on the way into it
// (palu_paged4_append) and back out of it (palu_paged4_read).
//
// A CTA has the 16 tokens of a block, aligned in the cache, of up to four heads
// of keys or values, a half-warp a token, a lane eight consecutive channels, so
// that four lanes are a group and its minimum and maximum take two shuffles.
// Transformed keys pass once through shared memory from the rotation's order
// of channels.  A token's key codes are 64 contiguous bytes of the block; its
// value codes are every sixteenth byte or so, because the attention takes a
// word's eight codes as a product's operand.  So a block's value codes are put
// together in shared memory and go out as whole words, or, where the call does
// not bring all of a word's tokens, as the bytes that it does bring.  Queries
// take the same path as in the uncompressed cache, in CTAs of their own, which
// wait for memory while those of keys and values compute: so the two kinds
// alternate in the grid.  Issue slots bound it (75 %): 9,790 tokens of 24 query and
// 8 KV heads 42 us, 173 MB of rows and codes; reading them back 12 us.
#include <math.h>

#include "paged4.cuh"
#include "qk_transform.cuh"

namespace palu {

// Smaller and larger of two pairs of elements, NaN if either is.
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The word of a lane's eight codes: code i in bits 4 i .. 4 i + 3, or, PAIRED, the
// even codes in its low half and the odd ones in the high half.  Codes are added
// up in fp32, four in the low 16 bits of a number from 2^23 on.
template <bool PAIRED>
struct CodeSum {
  float part[2] = {8388608.f, 8388608.f};
  __device__ __forceinline__ void add(int i, float c) {
    constexpr float kWeight[4] = {1.f, 16.f, 256.f, 4096.f};
    float& to = part[PAIRED ? i & 1 : i >> 2];
    to = fmaf(c, kWeight[PAIRED ? i >> 1 : i & 3], to);
  }
  __device__ __forceinline__ uint32_t word() const {
    return __byte_perm(__float_as_uint(part[0]), __float_as_uint(part[1]), 0x5410);
  }
};
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
// By a division a channel.  (Out of line: it is rarely wanted, and its code is long.)
template <bool BF16, bool PAIRED>
__device__ __noinline__ uint32_t divide8(uint4 raw, float s, float z) {
  float x[8];
  unpack8<BF16>(raw, x);
  CodeSum<PAIRED> sum;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    sum.add(i, s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], z), s)), 0.f), 15.f) : 0.f);
  return sum.word();
}

// The codes of a lane's eight channels, and the group's scale and zero.
//   rint((x - z) / s), cut to 0 .. 15, without a division a channel: with r near
// 1 / (15.49 s), v = (x - z) r saturated to 0 .. 1 and y = 15.49 v are within
// 1e-5 of the quotient (six roundings of 2^-24, one of them twice that, at up to
// 15.5) where that is in range, and y + 1.5 2^23 rounds to the nearest even
// integer.  Only where y lies within 1e-5 of a border between two codes does the
// rounded quotient decide.  (max - min) / 15 is its product with 1 / 15 and one
// step of correction, which gives the rounded quotient for every significand.
// With a division each the append of 9,790 tokens took 67 us, 59 % of the ALU's
// slots.
template <bool BF16, bool PAIRED>
__device__ __forceinline__ uint32_t quantise8(const uint4& raw, unsigned mask, uint16_t* scale, uint16_t* zero) {
  uint32_t mn = min2<BF16>(min2<BF16>(raw.x, raw.y), min2<BF16>(raw.z, raw.w));
  uint32_t mx = max2<BF16>(max2<BF16>(raw.x, raw.y), max2<BF16>(raw.z, raw.w));
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    mn = min2<BF16>(mn, __shfl_xor_sync(mask, mn, m));
    mx = max2<BF16>(mx, __shfl_xor_sync(mask, mx, m));
  }
  mn = min2<BF16>(mn, __byte_perm(mn, 0, 0x1032));
  mx = max2<BF16>(mx, __byte_perm(mx, 0, 0x1032));
  float lo = unpack2<BF16>(mn).x, hi = unpack2<BF16>(mx).x;
  if (!(lo > -INFINITY && hi < INFINITY)) {  // NaN among them too
    *scale = 0;
    *zero = 0x7e00;
    return 0;
  }
  if (BF16) {
    lo = fminf(fmaxf(lo, -65504.f), 65504.f);
    hi = fminf(fmaxf(hi, -65504.f), 65504.f);
  }
  const float range = __fsub_rn(hi, lo), q = __fmul_rn(range, 1.f / 15.f);
  __half s = __float2half_rn(fmaf(fmaf(-15.f, q, range), 1.f / 15.f, q));
  const __half z = __float2half_rn(lo);
  const float zf = __half2float(z);
  // a step less where the largest code would stand for more than fp16 has
  if (fmaf(15.f, __half2float(s), zf) > 65504.f) s = __ushort_as_half(__half_as_ushort(s) - 1);
  const float sf = __half2float(s);
  *scale = __half_as_ushort(s);
  *zero = __half_as_ushort(z);
  float x[8];
  unpack8<BF16>(raw, x);
  constexpr float kTop = 15.49f, kRound = 12582912.f;
  const float r = sf > 0.f ? __fdividef(1.f / kTop, sf) : 0.f;
  CodeSum<PAIRED> sum;
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v;  // saturated in the product itself
    asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(v) : "f"(__fsub_rn(x[i], zf)), "f"(r));
    const float c = __fadd_rn(fmaf(v, kTop, kRound), -kRound);
    off = fmaxf(off, fabsf(fmaf(v, kTop, -c)));
    sum.add(i, c);
  }
  return off > 0.5f - 1e-5f ? divide8<BF16, PAIRED>(raw, sf, zf) : sum.word();
}

// Key codes back from the word that has the odd channels in its high half.
__device__ __forceinline__ uint32_t key_codes(uint32_t w) {
  uint32_t even = w & 0xffffu, odd = w >> 16;
  even = (even | even << 8) & 0x00ff00ffu;
  odd = (odd | odd << 8) & 0x00ff00ffu;
  even = (even | even << 4) & 0x0f0f0f0fu;
  odd = (odd | odd << 4) & 0x0f0f0f0fu;
  return even | odd << 4;
}

// Where token t of a block has its value codes (of lane l's channels, the byte
// of g = 0) and its scale of a group.
__device__ __forceinline__ int value_byte(int t, int l) {
  return 512 * (l >> 3) + 16 * ((t & 7) >> 1) + 4 * ((l >> 1) & 3) + 2 * (t & 1) + (t >> 3);
}
__device__ __forceinline__ int value_scale(int t, int group) {
  return ((((t & 7) >> 1) * 2 + (t >> 3)) * 4 + group) * 4 + 2 * (t & 1);
}

struct Append4Params {
  QkParams q;             // with the operands of keys and values
  unsigned long long kv;  // CTAs of keys and values, of all, in 2^-32, rounded up
  int kv_runs;
};

template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads, 5) paged4_append_kernel(const Append4Params a) {
  const QkParams& p = a.q;
  __shared__ __align__(16) uint8_t stage[kRunHeads * (kBlock4 - kValueCodes4)];
  __shared__ __align__(16) uint16_t turned[kAppendThreads / 16][kHeadDim];
  __shared__ unsigned live_s;
  // CTAs of keys and values before this one; whether it is one
  const int y = (int)(blockIdx.x * a.kv >> 32);
  if ((int)((blockIdx.x + 1) * a.kv >> 32) == y) {
    const int z = (int)blockIdx.x - y, tile = z / p.q_runs;
    transform_tile<BF16, INTERLEAVED, true>(p, tile, z - tile * p.q_runs);
    return;
  }
  const int x = y / (2 * a.kv_runs), run = y - x * 2 * a.kv_runs;
  const bool values = run >= a.kv_runs;
  const int h0 = (values ? run - a.kv_runs : run) * kRunHeads, nh = min(kRunHeads, p.hk - h0);
  const int t = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const unsigned mask = (threadIdx.x & 16) ? 0xffff0000u : 0x0000ffffu;
  BlockWork w;
  if (threadIdx.x == 0) live_s = 0;
  if (!block_work(p.c, p.offsets, nullptr, p.rows, x, run == 0, &w)) return;
  // the token's place in the rotation; without one it is not appended, neither keys nor values
  float4 co = {}, si = {};
  const bool pairs = lane < (p.tr.rope_dim >> 3);
  if (p.tr.cos_sin != nullptr && w.live) {
    const long long pos = p.positions ? __ldg(p.positions + w.row) : w.place;
    if (pos < 0 || pos >= p.tr.n_positions) {
      w.live = false;
      if (lane == 0) atomicOr(p.c.error, PALU_DEVERR_POSITION);
    } else if (!values && pairs) {
      const float* cs = p.tr.cos_sin + pos * p.tr.rope_dim + 4 * lane;
      co = __ldg(reinterpret_cast<const float4*>(cs));
      si = __ldg(reinterpret_cast<const float4*>(cs + (p.tr.rope_dim >> 1)));
    }
  }
  if (!values) {
    if (!w.live) return;  // no barrier of the CTA from here on
    const int ca = !INTERLEAVED && pairs ? 4 * lane : 8 * lane;
    const int cb = !INTERLEAVED && pairs ? (p.tr.rope_dim >> 1) + 4 * lane : 8 * lane + 4;
    const uint16_t* src = p.k + w.row * p.ks1 + h0 * p.ks2;
    // the loop over the heads is kept rolled, a load ahead: four times its code is more than the instruction cache likes
    uint2 lo, hi;
    auto load = [&](int i) {
      lo = __ldg(reinterpret_cast<const uint2*>(src + i * p.ks2 + ca));
      hi = __ldg(reinterpret_cast<const uint2*>(src + i * p.ks2 + cb));
    };
    load(0);
    uint8_t* block = block_of_work(p.c, w);
    if (!block) return;
    block += h0 * p.c.ks1;
    const uint16_t* wsrc = static_cast<const uint16_t*>(p.tr.k_weight);
    float wt[8] = {};
    if (wsrc) {
      const uint2 wl = __ldg(reinterpret_cast<const uint2*>(wsrc + ca)), wh = __ldg(reinterpret_cast<const uint2*>(wsrc + cb));
      const uint32_t raw[4] = {wl.x, wl.y, wh.x, wh.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(raw[i]);
        wt[2 * i] = f.x;
        wt[2 * i + 1] = f.y;
      }
    }
#pragma unroll 1
    for (int i = 0; i < nh; ++i) {
      uint2 a = lo, b = hi;
      if (i + 1 < nh) load(i + 1);
      transform_row<BF16, INTERLEAVED>(a, b, wsrc != nullptr, wt, pairs && p.tr.cos_sin != nullptr, co, si, p.tr.eps, mask);
      *reinterpret_cast<uint2*>(&turned[t][ca]) = a;
      *reinterpret_cast<uint2*>(&turned[t][cb]) = b;
      __syncwarp(mask);
      const uint4 raw = *reinterpret_cast<const uint4*>(&turned[t][8 * lane]);
      __syncwarp(mask);
      uint16_t s, z;
      const uint32_t codes = quantise8<BF16, true>(raw, mask, &s, &z);
      uint8_t* to = block + i * p.c.ks1;
      *reinterpret_cast<uint32_t*>(to + 64 * t + 16 * (lane & 3) + 4 * (lane >> 2)) = codes;
      if ((lane & 3) == 0) {
        uint16_t* sz = reinterpret_cast<uint16_t*>(to + kKeyScales4 + 16 * t) + (lane >> 2);
        sz[0] = s;
        sz[4] = z;
      }
    }
    return;
  }
  // values: the block's image
  const uint16_t* const src = p.v + (w.live ? w.row : 0) * p.vs1 + h0 * p.vs2 + 8 * lane;
  uint4 next = {};
  if (w.live) next = __ldg(reinterpret_cast<const uint4*>(src));
  uint8_t* block = block_of_work(p.c, w);
  if (!block) return;
  block += h0 * p.c.ks1;
  __syncthreads();
  if (w.live) {
    if (lane == 0) atomicOr(&live_s, 1u << t);
#pragma unroll 1
    for (int i = 0; i < nh; ++i) {
      const uint4 raw = next;
      if (i + 1 < nh) next = __ldg(reinterpret_cast<const uint4*>(src + (i + 1) * p.vs2));
      uint16_t s, z;
      const uint32_t mine = quantise8<BF16, false>(raw, mask, &s, &z), other = __shfl_xor_sync(mask, mine, 1);
      uint8_t* const im = stage + i * (kBlock4 - kValueCodes4);
      // an even lane and the odd one behind it have the two nibbles of eight bytes: it writes those of g 0, 2, 4, 6, the
      // odd one the others
      const uint32_t bytes = lane & 1 ? (mine & 0xf0f0f0f0u) | (other >> 4 & 0x0f0f0f0fu) : (mine & 0x0f0f0f0fu) | (other & 0x0f0f0f0fu) << 4;
      uint8_t* const to = im + value_byte(t, lane) + 64 * (lane & 1);
#pragma unroll
      for (int g = 0; g < 4; ++g) to[128 * g] = (uint8_t)(bytes >> (8 * g));
      if ((lane & 3) == 0) {
        uint8_t* sz = im + 1024 + value_scale(t, lane >> 2);
        *reinterpret_cast<uint16_t*>(sz) = s;
        *reinterpret_cast<uint16_t*>(sz + 128) = z;
      }
    }
  }
  __syncthreads();
  const unsigned live = live_s;
  if (live == 0xffffu) {
    constexpr int kPieces = (kBlock4 - kValueCodes4) / 16;
    for (int i = threadIdx.x; i < nh * kPieces; i += kAppendThreads) {
      const int h = i / kPieces;
      *reinterpret_cast<uint4*>(block + h * p.c.ks1 + kValueCodes4 + 16 * (i - h * kPieces)) = *reinterpret_cast<const uint4*>(stage + 16 * i);
    }
    return;
  }
  constexpr int kWords = (kBlock4 - kValueCodes4) / 4;
  for (int i = threadIdx.x; i < nh * kWords; i += kAppendThreads) {
    const int h = i / kWords, k = i - h * kWords;
    const uint8_t* im = stage + 4 * i;
    uint8_t* to = block + h * p.c.ks1 + kValueCodes4 + 4 * k;
    // the word's tokens, two bytes each of one or one byte each of four
    const bool sc = k >= 256;
    const int c = sc ? (k >> 3) & 3 : (k >> 2) & 3, t0 = 2 * c + (sc ? 8 * ((k >> 2) & 1) : 0);
    const unsigned want = sc ? 3u << t0 : 0x0303u << t0;
    if ((live & want) == want) {
      *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(im);
    } else if (live & want) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int tok = sc ? t0 + (b >> 1) : t0 + (b >> 1) + 8 * (b & 1);
        if (live >> tok & 1) to[b] = im[b];
      }
    }
  }
}

struct Read4Params {
  PagedView c;
  const int* offsets;
  const long long* starts;
  uint16_t *k_out, *v_out;
  long long rows;
  int kv_runs;
};

// z + s c of a lane's eight channels, rounded.
template <bool BF16>
__device__ __forceinline__ uint4 values8(uint32_t codes, float s, float z) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = pack2<BF16>(fmaf(s, (float)(codes >> (8 * i) & 15), z), fmaf(s, (float)(codes >> (8 * i + 4) & 15), z));
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) paged4_read_kernel(const Read4Params p) {
  __shared__ __align__(16) uint8_t blocks[kRunHeads * kBlock4];
  const int x = blockIdx.x / p.kv_runs, run = blockIdx.x - x * p.kv_runs;
  const int h0 = run * kRunHeads, nh = min(kRunHeads, p.c.kv_heads - h0);
  BlockWork w;
  if (!block_work(p.c, p.offsets, p.starts, p.rows, x, run == 0, &w)) return;
  const uint8_t* const block = block_of_work(p.c, w);
  if (!block) return;
  for (int i = threadIdx.x; i < nh * (kBlock4 / 16); i += kAppendThreads) {
    const int h = i / (kBlock4 / 16), k = i - h * (kBlock4 / 16);
    *reinterpret_cast<uint4*>(blocks + 16 * i) = __ldg(reinterpret_cast<const uint4*>(block + (h0 + h) * p.c.ks1) + k);
  }
  __syncthreads();
  if (!w.live) return;
  const int t = threadIdx.x >> 4, lane = threadIdx.x & 15;
  for (int i = 0; i < nh; ++i) {
    const uint8_t* b = blocks + i * kBlock4;
    const long long at = ((long long)w.row * p.c.kv_heads + h0 + i) * kHeadDim + 8 * lane;
    const __half* sz = reinterpret_cast<const __half*>(b + kKeyScales4 + 16 * t) + (lane >> 2);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(b + 64 * t + 16 * (lane & 3) + 4 * (lane >> 2));
    *reinterpret_cast<uint4*>(p.k_out + at) = values8<BF16>(key_codes(kw), __half2float(sz[0]), __half2float(sz[4]));
    uint32_t vw = 0;
    const uint8_t* vb = b + kValueCodes4 + value_byte(t, lane);
#pragma unroll
    for (int g = 0; g < 8; ++g) vw |= (uint32_t)(vb[64 * g] >> (4 * (lane & 1)) & 15) << (4 * g);
    const uint8_t* vs = b + kValueScales4 + value_scale(t, lane >> 2);
    *reinterpret_cast<uint4*>(p.v_out + at) = values8<BF16>(vw, __half2float(*reinterpret_cast<const __half*>(vs)),
                                                            __half2float(*reinterpret_cast<const __half*>(vs + 128)));
  }
}

palu_status paged4_check(const palu_paged4_cache* c) {
  if (!c) return fail(PALU_ERR_INVALID_ARG, "cache is NULL");
  if (c->magic != kPaged4Magic) return fail(PALU_ERR_NOT_INITIALIZED, "paged cache is not initialised");
  return PALU_OK;
}

static bool bytes_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_paged4_cache_init(palu_paged4_cache* cache, int32_t dtype, int32_t kv_heads, int32_t page_size,
                                              int64_t n_pages, void* pages, const int64_t strides[2],
                                              const int32_t* page_table, int64_t batch, int64_t table_width,
                                              const int64_t* lengths, uint32_t* error) {
  if (!cache) return fail(PALU_ERR_INVALID_ARG, "cache is NULL");
  cache->magic = 0;
  if (dtype != PALU_TYPE_F16 && dtype != PALU_TYPE_BF16) return fail(PALU_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(PALU_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (kv_heads < 1 || kv_heads > 65536 || n_pages < 1 || n_pages > 0x7fffffff)
    return fail(PALU_ERR_INVALID_ARG, "bad head or page count");
  if (batch < 1 || table_width < 1) return fail(PALU_ERR_INVALID_ARG, "batch and table_width must be positive");
  if (batch > kMaxPagedBatch) return fail(PALU_ERR_UNSUPPORTED, "at most 4096 sequences");
  if (table_width > (1LL << 30) / page_size) return fail(PALU_ERR_UNSUPPORTED, "at most 2^30 tokens a sequence");
  if (!pages || !strides || !page_table || !lengths || !error) return fail(PALU_ERR_INVALID_ARG, "NULL pointer");
  if ((uintptr_t)pages & 15) return fail(PALU_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  for (int i = 0; i < 2; ++i)
    if (strides[i] < 16 || strides[i] % 16 || strides[i] >= (1LL << 39))
      return fail(PALU_ERR_INVALID_ARG, "page strides must be positive multiples of 16 bytes (and less than 2^39)");
  if (n_pages > (1LL << 56) / strides[0] || kv_heads > (1LL << 56) / strides[1])
    return fail(PALU_ERR_INVALID_ARG, "the pool is larger than 2^56 bytes");
  if (((uintptr_t)page_table | (uintptr_t)error) & 3 || (uintptr_t)lengths & 7)
    return fail(PALU_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  cache->dtype = dtype;
  cache->kv_heads = kv_heads;
  cache->page_size = page_size;
  cache->batch = (int32_t)batch;
  cache->table_width = (int32_t)table_width;
  cache->n_pages = n_pages;
  cache->pages = pages;
  cache->strides[0] = strides[0];
  cache->strides[1] = strides[1];
  cache->page_table = page_table;
  cache->lengths = lengths;
  cache->error = error;
  cache->magic = kPaged4Magic;
  return PALU_OK;
}

extern "C" palu_status palu_paged4_append(const palu_paged4_cache* cache, const palu_qk_transform* transform,
                                          int64_t tokens, const int32_t* offsets, int32_t q_heads, const void* q,
                                          const int64_t q_strides[2], const void* k, const int64_t k_strides[2],
                                          const void* v, const int64_t v_strides[2], const int64_t* positions,
                                          void* q_out, void* stream) {
  palu_status st = paged4_check(cache);
  if (st != PALU_OK || (st = transform_check(transform)) != PALU_OK) return st;
  if (tokens < 1 || tokens > 0x7fffffff) return fail(PALU_ERR_INVALID_ARG, "tokens must be in [1, 2^31)");
  if (q_heads < 0 || q_heads > 65536 || (q_heads > 0) != (q != nullptr) || (q_heads > 0) != (q_out != nullptr))
    return fail(PALU_ERR_INVALID_ARG, "q, q_out and q_heads come together");
  if (!offsets || ((uintptr_t)offsets & 3)) return fail(PALU_ERR_INVALID_ARG, "offsets must be given, 4-byte aligned");
  if (q && (st = rows_check("q", q, q_strides, 2)) != PALU_OK) return st;
  if ((st = rows_check("k", k, k_strides, 2)) != PALU_OK || (st = rows_check("v", v, v_strides, 2)) != PALU_OK) return st;
  if ((uintptr_t)q_out & 15) return fail(PALU_ERR_INVALID_ARG, "q_out must be 16-byte aligned");
  if ((uintptr_t)positions & 7) return fail(PALU_ERR_INVALID_ARG, "positions must be 8-byte aligned");
  const int64_t qe[2] = {tokens, q_heads}, ke[2] = {tokens, cache->kv_heads};
  if (q && (rows_overlap(q_out, tokens * q_heads, q, q_strides, qe, 2) || rows_overlap(q_out, tokens * q_heads, k, k_strides, ke, 2) ||
            rows_overlap(q_out, tokens * q_heads, v, v_strides, ke, 2)))
    return fail(PALU_ERR_INVALID_ARG, "q_out overlaps an input");
  Append4Params a = {};
  QkParams& p = a.q;
  p.tr = *transform;
  if (!p.tr.cos_sin) p.tr.rope_dim = 0;  // no pairs
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  if (q) p.qs1 = q_strides[0], p.qs2 = q_strides[1];
  p.ks1 = k_strides[0], p.ks2 = k_strides[1];
  p.vs1 = v_strides[0], p.vs2 = v_strides[1];
  p.positions = reinterpret_cast<const long long*>(positions);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.error = cache->error;
  p.rows = tokens;
  p.tokens = tokens;
  p.hq = q_heads;
  p.hk = cache->kv_heads;
  p.q_runs = (q_heads + kRunHeads - 1) / kRunHeads;
  p.offsets = offsets;
  p.c = paged4_view(cache);
  a.kv_runs = (cache->kv_heads + kRunHeads - 1) / kRunHeads;
  const long long q_ctas = (tokens + kAppendThreads / 16 - 1) / (kAppendThreads / 16) * p.q_runs;
  const long long kv_ctas = (tokens / 16 + 2LL * cache->batch) * 2 * a.kv_runs, grid = q_ctas + kv_ctas;
  if (grid > 0x7fffffff) return fail(PALU_ERR_UNSUPPORTED, "too many rows for one call");
  // rounded up: of i CTAs floor(i kv / 2^32) are of keys and values, and of all of them kv_ctas, as grid < 2^32
  a.kv = (((unsigned long long)kv_ctas << 32) + grid - 1) / grid;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = cache->dtype == PALU_TYPE_BF16, inter = p.tr.interleaved != 0;
  auto* const kernel = bf16 ? inter ? paged4_append_kernel<true, true> : paged4_append_kernel<true, false>
                            : inter ? paged4_append_kernel<false, true> : paged4_append_kernel<false, false>;
  kernel<<<(unsigned)grid, kAppendThreads, 0, s>>>(a);
  return cuda_check(cudaGetLastError(), "paged4_append_kernel launch");
}

extern "C" palu_status palu_paged4_read(const palu_paged4_cache* cache, int64_t tokens, const int32_t* offsets,
                                        const int64_t* starts, void* k_out, void* v_out, void* stream) {
  palu_status st = paged4_check(cache);
  if (st != PALU_OK) return st;
  if (tokens < 1 || tokens > 0x7fffffff) return fail(PALU_ERR_INVALID_ARG, "tokens must be in [1, 2^31)");
  if (!offsets || ((uintptr_t)offsets & 3)) return fail(PALU_ERR_INVALID_ARG, "offsets must be given, 4-byte aligned");
  if ((uintptr_t)starts & 7) return fail(PALU_ERR_INVALID_ARG, "starts must be 8-byte aligned");
  if (!k_out || !v_out || (((uintptr_t)k_out | (uintptr_t)v_out) & 15))
    return fail(PALU_ERR_INVALID_ARG, "k_out and v_out must be given, 16-byte aligned");
  const int64_t bytes = tokens * cache->kv_heads * kHeadDim * 2;
  const int64_t pool = (cache->n_pages - 1) * cache->strides[0] + (cache->kv_heads - 1) * cache->strides[1] +
                       (int64_t)cache->page_size / 16 * kBlock4;
  if (bytes_meet(k_out, bytes, v_out, bytes)) return fail(PALU_ERR_INVALID_ARG, "k_out overlaps v_out");
  if (bytes_meet(k_out, bytes, cache->pages, pool) || bytes_meet(v_out, bytes, cache->pages, pool))
    return fail(PALU_ERR_INVALID_ARG, "an output overlaps the pages");
  Read4Params p = {};
  p.c = paged4_view(cache);
  p.offsets = offsets;
  p.starts = reinterpret_cast<const long long*>(starts);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.rows = tokens;
  p.kv_runs = (cache->kv_heads + kRunHeads - 1) / kRunHeads;
  const long long grid = (tokens / 16 + 2LL * cache->batch) * p.kv_runs;
  if (grid > 0x7fffffff) return fail(PALU_ERR_UNSUPPORTED, "too many rows for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->dtype == PALU_TYPE_BF16)
    paged4_read_kernel<true><<<(unsigned)grid, kAppendThreads, 0, s>>>(p);
  else
    paged4_read_kernel<false><<<(unsigned)grid, kAppendThreads, 0, s>>>(p);
  return cuda_check(cudaGetLastError(), "paged4_read_kernel launch");
}

extern "C" palu_status palu_paged4_sync(const palu_paged4_cache* cache, uint32_t* device_error, void* stream) {
  palu_status st = paged4_check(cache);
  if (st != PALU_OK) return st;
  palu_paged_cache c = {};  // the error word is the same
  c.magic = kPagedMagic;
  c.error = cache->error;
  return palu_paged_sync(&c, device_error, stream);
}
