/*
 * bit_grouped_expert_moe_gb300 — C ABI of rotary positions for NVIDIA GB300
 * (sm_103a): queries and keys normed per head (optionally) and rotated by
 * their tokens' positions in one pass over the data. What the attention calls
 * (attention.h, kv8.h, paged.h) take as q and k is what this call writes.
 *
 * Per head x of D values, at position p:
 *   norm (optional)  x <- x / sqrt(mean(x^2) + eps) * (gain_offset + gain)
 *   rotation         the first `rot` values form rot / 2 pairs (a, b); pair i
 *                    turns by the angle p w_i:
 *                      a <- m (a cos(p w_i) - b sin(p w_i))
 *                      b <- m (b cos(p w_i) + a sin(p w_i))
 *                    the other values pass through. m is `magnitude`.
 *   Pairs: MOE_ROPE_HALF   (x[i], x[i + rot / 2])
 *          MOE_ROPE_PAIRS  (x[2 i], x[2 i + 1])
 *
 * Angles are kept in turns: a table holds w_i / 2 pi modulo 1 as a 64-bit
 * fixed-point number, and p times it, modulo 2^64, is the turn of position p,
 * exact but for the table's own rounding (2^-54 of a turn for |w_i| <= 1, so
 * 2^-23 at p = 2^31). A far position loses nothing to a near one.
 *
 * Numerics: bf16 in and out, fp32 between, rounded once. A turn goes to fp32
 * with an error of up to 2^-26 of a turn, sine and cosine to fp32. The mean
 * square of any finite head is formed without overflow. A head that holds
 * infinities or NaN comes out with NaN in what they reach.
 *
 * Ownership, streams and errors as in moe.h: device pointers owned by the
 * caller, host shape and spec pointers, no allocation, no host
 * synchronisation, all work on `stream`.
 */
#ifndef BGMOE_ROPE_H
#define BGMOE_ROPE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_rope_scaling {
  MOE_ROPE_PLAIN = 0,  /* w */
  MOE_ROPE_LINEAR = 1, /* w / factor: positions interpolated */
  MOE_ROPE_BANDS = 2,  /* by the turns t = original w / 2 pi of the original context: w / factor for t <= low, w for
                          t >= high, in between w / factor + (w - w / factor) (t - low) / (high - low) */
  MOE_ROPE_RAMP = 3    /* "YaRN" (Peng et al. 2023): by the index i, with d(t) = rot ln(original / (2 pi t)) / (2 ln base),
                          lo = max(floor(d(high)), 0), hi = min(ceil(d(low)), rot - 1) and u = (i - lo) / max(hi - lo,
                          0.001) clamped to 0..1: w (1 - u) + (w / factor) u; magnitude 0.1 ln(factor) + 1 */
} moe_rope_scaling;

typedef enum moe_rope_layout { MOE_ROPE_HALF = 0, MOE_ROPE_PAIRS = 1 } moe_rope_layout;

#define MOE_ROPE_NORM_Q 1
#define MOE_ROPE_NORM_K 2

/* How frequencies are formed (host side). */
typedef struct moe_rope_frequencies {
  int32_t rot;         /* values per head that turn: a multiple of 16, 16 .. 256 */
  int32_t scaling;     /* moe_rope_scaling */
  int32_t original;    /* positions of the original context (bands, ramp): >= 1 */
  int32_t reserved;    /* 0 */
  double base;         /* w_i = base^(-2 i / rot): > 1 */
  double factor;       /* >= 1 */
  double low, high;    /* turns (bands, ramp): 0 < low < high */
  const double* given; /* [rot / 2] host: radians per position in place of base^(-2 i / rot), or NULL. Finite */
} moe_rope_frequencies;

/* Fills turns[0 .. rot / 2) (host memory; copy it to the device) and the
 * magnitude that goes with the scaling. No CUDA call. */
moe_status moe_rope_table(const moe_rope_frequencies* f, uint64_t* turns, float* magnitude);

/* How heads are normed and rotated. */
typedef struct moe_rope_spec {
  const uint64_t* turns; /* device [rot / 2], 16-byte aligned; NULL if rot = 0 */
  const void* q_gain;    /* device bf16 [D], 16-byte aligned, or NULL: gain_offset + gain is 1 */
  const void* k_gain;
  int32_t rot;           /* 0 (no rotation) or a multiple of 16, <= D */
  int32_t layout;        /* moe_rope_layout */
  int32_t norm;          /* MOE_ROPE_NORM_Q | MOE_ROPE_NORM_K */
  float eps;             /* finite; with a norm at least 1e-30 */
  float gain_offset;     /* finite */
  float magnitude;       /* finite */
} moe_rope_spec;

/* Shape of one call. Supported: 0 <= T <= 2^24; 0 <= Hq, Hk <= 4096, not both
 * 0, T * (Hq + Hk) <= 2^30; D a multiple of 16, 16 .. 256. Strides: elements from token
 * to token, 0 for packed tokens, or a multiple of 8 of at least one token's
 * (Hq D, Hk D). */
typedef struct moe_rope_shape {
  int32_t T;         /* tokens */
  int32_t Hq;        /* query heads (0: no queries) */
  int32_t Hk;        /* key heads (0: no keys) */
  int32_t D;         /* head size */
  int32_t q_stride;  /* of q */
  int32_t k_stride;  /* of k */
  int32_t qo_stride; /* of q_out */
  int32_t ko_stride; /* of k_out */
} moe_rope_shape;

/* q, q_out bf16 [T][Hq][D], k, k_out bf16 [T][Hk][D], 16-byte aligned;
 * positions int32 [T], any value; NULL with rot = 0. q_out may be q and k_out
 * k (with the same stride); outputs must not overlap inputs otherwise. T == 0
 * is a no-op. */
moe_status moe_rope(const moe_rope_shape* shape, const moe_rope_spec* spec, const void* q, const void* k,
                    const int32_t* positions, void* q_out, void* k_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BGMOE_ROPE_H */
