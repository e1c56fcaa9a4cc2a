/*
 * libpalu — the rotation tables that palu_qk_transform takes, plain or scaled
 * for contexts longer than those of the training.
 *
 * The caches take rotated keys (page "PALU — True Low-Rank Latent Storage for
 * Keys and Values", "How it works": the cache sits behind the rotation); the
 * 131072-token workload is beyond most models' training length.
 *
 * Conventions are those of palu.h.
 */
#ifndef PALU_ROPE_H
#define PALU_ROPE_H

#include "palu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pair i of d / 2 (d = rope_dim) turns by f_i a position, f_i = base^(-2i/d):
 *   PLAIN   f_i
 *   LINEAR  f_i / factor (position interpolation)
 *   NTK     f_i with base * factor^(d / (d-2)): the fastest pair keeps its
 *           turn, the slowest is stretched by factor
 *   PARTS   f_i (t + (1 - t) / factor), with the turns r = original f_i / 2 pi
 *           of the pair in the context of the training and
 *           t = min(max((r - low_turns) / (high_turns - low_turns), 0), 1).
 *           The ramp runs over the turns, which is over original / wavelength: a
 *           model that states it so, without a magnitude, is this kind with magnitude
 *           1 (low_turns 1 and high_turns 4, say).  A ramp that runs over the pair's
 *           number i, and frequencies given one by one, are none of these. */
enum { PALU_ROPE_PLAIN = 0, PALU_ROPE_LINEAR = 1, PALU_ROPE_NTK = 2, PALU_ROPE_PARTS = 3 };

typedef struct {
  int32_t kind;
  int32_t rope_dim;      /* a multiple of 16, 16 .. 128 */
  double base;           /* > 1 */
  double factor;         /* >= 1; not read for PLAIN */
  double original;       /* PARTS: tokens of the training's context, > 0 */
  double low_turns;      /* PARTS: 0 <= low_turns < high_turns */
  double high_turns;
  double magnitude;      /* the cosines and sines are multiplied by it; finite in fp32 */
} palu_rope_scaling;

/* Row r of the table, r in 0 .. positions - 1: the cosines, then the sines, of
 * (start + r) f_i, times magnitude.  Angles are reduced in whole numbers (f_i /
 * 2 pi as a 64-bit fraction of a turn): they are off by 2^-64 of a turn a position
 * at most (bases up to 10^300), a value by 2^-22 of magnitude more.
 *   out    device fp32 [positions, rope_dim], contiguous, 16-byte aligned.
 *   start  0 .. 2^40.  positions 0 .. 2^31 - 1.
 * One kernel launch. */
palu_status palu_rope_table(const palu_rope_scaling* scaling, int64_t start, int64_t positions, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PALU_ROPE_H */
