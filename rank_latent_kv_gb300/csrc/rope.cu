// Rotation tables (include/rope.h).
//
// A table is written once and read by every layer; 131,072 positions of 128
// are 67 MB, so writing them is the bound if a value costs few instructions.
// The angles of far positions are the difficulty: p f_i needs more bits than
// fp32 has, and fp64 arithmetic is 1/60 of fp32's rate here.  So a pair's turn a
// position, f_i / 2 pi, is a 64-bit fraction of a whole turn, and its product
// with the position wraps around exactly: two integer additions from one row to
// the next.  The host finds those fractions in sums of two doubles: in one double each
// an exponent's rounding times ln base, and those of the powers, made 2^-48 of the
// angle, 2^-8 at 2^40 positions.  Of the fraction the nearest quarter turn is taken off, and the rest,
// at most an eighth of a turn, goes through the Taylor series of sine (to the
// 9th power, off by 2e-9) and cosine (to the 10th, 1e-10).  131,072 positions of
// 128: 11.1 us, 6.0 TB/s.
#include <math.h>

#include "palu_internal.cuh"
#include "rope.h"

namespace palu {

struct RopeParams {
  uint64_t turn[kHeadDim / 2];  // f_i / 2 pi in 2^-64 of a turn
  float* out;
  long long start, positions;
  float magnitude;
  int rope;
};

constexpr int kRopeThreads = 256;

// cos and sin of `turn` / 2^64 turns, times m
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, float m, float& co, float& si) {
  // an eighth of a turn more: the quarter turns, rounded, in the top two bits, the rest of the turn behind them; 32
  // bits of it are enough for angles to 2^-33
  const uint32_t near = (uint32_t)(turn >> 32) + (1u << 29);
  const int rest = (int)(__funnelshift_l((uint32_t)turn, near, 2) ^ 0x80000000u);
  const float x = (float)rest * (6.28318530717958648f * 0x1p-34f), u = x * x;
  const float s = x * fmaf(u, fmaf(u, fmaf(u, fmaf(u, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), 1.f);
  const float c = fmaf(u, fmaf(u, fmaf(u, fmaf(u, fmaf(u, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  // a quarter turn swaps the two; the cosine is negative in the second and third, the sine in the third and fourth
  const bool odd = near & (1u << 30);
  const uint32_t a = __float_as_uint((odd ? s : c) * m), b = __float_as_uint((odd ? c : s) * m);
  co = __uint_as_float(a ^ ((near ^ near << 1) & 0x80000000u));
  si = __uint_as_float(b ^ (near & 0x80000000u));
}

// A thread has four pairs and goes down the rows; rope_dim / 8 threads a row.
// All CTAs are resident: a second wave of the table's 131,072 rows is a third more time.
constexpr int kRopeCtas = 5;  // an SM
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_table_kernel(const __grid_constant__ RopeParams p) {
  const int per_row = p.rope >> 3;
  const long long t = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const long long step = (long long)gridDim.x * kRopeThreads / per_row;  // rows; threads behind them have none
  const int part = (int)(t % per_row);
  long long row = t / per_row;
  if (row >= step) return;
  uint64_t at[4], by[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    at[i] = (uint64_t)(p.start + row) * p.turn[4 * part + i];
    by[i] = (uint64_t)step * p.turn[4 * part + i];
  }
  for (; row < p.positions; row += step) {
    float co[4], si[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_cos_sin(at[i], p.magnitude, co[i], si[i]);
      at[i] += by[i];
    }
    float* to = p.out + row * p.rope + 4 * part;
    *reinterpret_cast<float4*>(to) = make_float4(co[0], co[1], co[2], co[3]);
    *reinterpret_cast<float4*>(to + (p.rope >> 1)) = make_float4(si[0], si[1], si[2], si[3]);
  }
}

// A number as the unevaluated sum of two doubles, hi the nearest: 2^-104 and a
// few roundings more an operation.
struct Sum2 {
  double hi, lo;
};
static Sum2 settle(double hi, double lo) {  // |hi| >= |lo|
  const double s = hi + lo;
  return {s, lo - (s - hi)};
}
static Sum2 add(Sum2 a, Sum2 b) {
  const double s = a.hi + b.hi, t = s - a.hi;
  return settle(s, (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo));
}
static Sum2 mul(Sum2 a, Sum2 b) {
  const double p = a.hi * b.hi;
  return settle(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
static Sum2 div(Sum2 a, Sum2 b) {
  const double q = a.hi / b.hi;
  const Sum2 r = add(a, mul({-q, 0.0}, b));
  return settle(q, r.hi / b.hi);
}
// x^(-1/n): pow's root and one step of Newton's method, 1 - (root^n - x) / (n x) times it.
static Sum2 inverse_root(double x, int n) {
  const Sum2 root = {pow(x, 1.0 / n), 0.0};
  Sum2 power = {1.0, 0.0}, square = root;
  for (int k = n; k; k >>= 1) {
    if (k & 1) power = mul(power, square);
    if (k > 1) square = mul(square, square);
  }
  const double off = add(power, {-x, 0.0}).hi / x / n;
  return div({1.0, 0.0}, fabs(off) < 1.0 ? mul(root, settle(1.0, -off)) : root);  // (it may overflow next to the largest x)
}

}  // namespace palu

using namespace palu;

extern "C" palu_status palu_rope_table(const palu_rope_scaling* scaling, int64_t start, int64_t positions, float* out,
                                       void* stream) {
  if (!scaling) return fail(PALU_ERR_INVALID_ARG, "scaling is NULL");
  const palu_rope_scaling& s = *scaling;
  const int d = s.rope_dim;
  if (d < 16 || d > kHeadDim || d % 16) return fail(PALU_ERR_UNSUPPORTED, "rope_dim must be a multiple of 16 in [16, 128]");
  if (s.kind < PALU_ROPE_PLAIN || s.kind > PALU_ROPE_PARTS) return fail(PALU_ERR_INVALID_ARG, "unknown kind of scaling");
  if (!(s.base > 1.0) || isinf(s.base)) return fail(PALU_ERR_INVALID_ARG, "base must be finite and above 1");
  if (s.kind != PALU_ROPE_PLAIN && (!(s.factor >= 1.0) || isinf(s.factor)))
    return fail(PALU_ERR_INVALID_ARG, "factor must be finite and at least 1");
  if (s.kind == PALU_ROPE_PARTS && (!(s.original > 0.0) || isinf(s.original) || !(s.low_turns >= 0.0) ||
                                    !(s.high_turns > s.low_turns) || isinf(s.high_turns)))
    return fail(PALU_ERR_INVALID_ARG, "original must be positive, and 0 <= low_turns < high_turns, all finite");
  if (!isfinite((float)s.magnitude)) return fail(PALU_ERR_INVALID_ARG, "magnitude must be finite");
  if (start < 0 || start > (1LL << 40) || positions < 0 || positions > 0x7fffffff)
    return fail(PALU_ERR_INVALID_ARG, "start must be in [0, 2^40], positions in [0, 2^31)");
  if (positions == 0) return PALU_OK;
  if (!out || ((uintptr_t)out & 15)) return fail(PALU_ERR_INVALID_ARG, "out must be given, 16-byte aligned");
  RopeParams p = {};
  const Sum2 one = {1.0, 0.0}, inv_two_pi = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};
  // f_1, to whose powers f_i belongs; of NTK base^(-2/d) factor^(-2/(d-2))
  Sum2 first = inverse_root(s.base, d / 2);
  if (s.kind == PALU_ROPE_NTK) first = mul(first, inverse_root(s.factor, d / 2 - 1));
  Sum2 f[kHeadDim / 2] = {one, first};
  for (int i = 2; i < d / 2; ++i) f[i] = i <= 8 ? mul(f[i - 1], first) : mul(f[i - 8], f[8]);  // (chains side by side)
  const Sum2 shrink = s.kind == PALU_ROPE_PLAIN ? one : div(one, {s.factor, 0.0});
  const Sum2 ramp = add({s.high_turns, 0.0}, {-s.low_turns, 0.0});
  for (int i = 0; i < d / 2; ++i) {
    Sum2 t = mul(f[i], inv_two_pi);  // turns a position
    if (s.kind == PALU_ROPE_LINEAR) t = mul(t, shrink);
    if (s.kind == PALU_ROPE_PARTS) {
      const Sum2 above = add(mul({s.original, 0.0}, t), {-s.low_turns, 0.0});
      if (above.hi <= 0.0) {
        t = mul(t, shrink);
      } else if (above.hi < ramp.hi) {
        const Sum2 part = div(above, ramp);
        t = mul(t, add(part, mul(add(one, {-part.hi, -part.lo}), shrink)));
      }
    }
    // below 2^62, to the nearest
    const double hi = ldexp(t.hi, 64);
    p.turn[i] = (uint64_t)hi;
    p.turn[i] += (int64_t)floor((hi - (double)p.turn[i]) + ldexp(t.lo, 64) + 0.5);
  }
  p.out = out;
  p.start = start;
  p.positions = positions;
  p.magnitude = (float)s.magnitude;
  p.rope = d;
  // at least one row a thread
  const long long threads = positions * (d >> 3), most = (long long)kRopeCtas * device_sm_count();
  const long long grid = (threads + kRopeThreads - 1) / kRopeThreads;
  rope_table_kernel<<<(unsigned)(grid < most ? grid : most), kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cuda_check(cudaGetLastError(), "rope_table_kernel launch");
}
