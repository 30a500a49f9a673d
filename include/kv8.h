/*
 * bit_grouped_expert_moe_gb300 — C ABI of an 8-bit KV cache for NVIDIA GB300
 * (sm_103a): new tokens' keys and values quantised into it as they are
 * written, ranges of it read back as bf16, and causal grouped-query attention
 * over it, from one query token per sequence (decode) to whole prompts.
 *
 * The cache holds one byte per value and one fp32 scale per (sequence, KV
 * head, block of `block` consecutive positions), for keys and for values
 * apart. A stored value is code * scale:
 *   MOE_KV8_INT8  code -127 .. 127, stored as the byte code + 128; the scale
 *                 of a block with largest magnitude a is fp32(a / 127);
 *   MOE_KV8_E4M3  code an e4m3 number (finite, |code| <= 448); the scale is
 *                 the smallest power of two with a / scale <= 448 (2^120 at
 *                 most, where codes stop at 240: 256 would be 2^128).
 * A scale is at least 2^-60, or 0 for a block of zeros only. Three bytes are
 * never stored: 0 in int8, which would be code -128, and 0x7F and 0xFF in
 * e4m3, which write and read take as +-480 and attention as NaN. Bytes past a
 * context may hold anything.
 *
 * Write: sequence b's new tokens go to positions starts[b], starts[b] + 1, ...
 *   A block that held no earlier token of the sequence takes the scale of its
 *   new values; one that did takes the larger of that and the scale it had
 *   (a scale never shrinks while its block fills). If the scale grew, the
 *   block's earlier codes are quantised again, from code * old scale. A code
 *   is x * fp32(1 / scale) rounded to nearest, ties to even. Repeating a
 *   sequence's last write changes nothing. Positions past the new tokens keep
 *   their bytes, but a write over earlier positions may leave their block
 *   another scale: what follows the new tokens in it is lost and has to be
 *   written again.
 *   Every finite input is allowed. A NaN is stored as 0 and an infinity as
 *   its sign times the largest finite magnitude of the block's new values,
 *   and MOE_ERR_RANGE is written to *status: the other values stay good.
 *
 * Read: the values of positions starts[b] .. of sequence b, the fp32 product
 *   code * scale rounded to bf16.
 *
 * Attention: the queries of sequence b are its last n = offsets[b+1] -
 *   offsets[b] positions; query i sees positions 0 .. lens[b] - n + i (its own
 *   key included):
 *     o[i,h,:] = sum_j softmax_j(scale * q[i,h,:] . K[b,g,j,:]) V[b,g,j,:],
 *     g = h / (Hq / Hkv).
 *   A query that sees no position (lens[b] < n, i < n - lens[b]) gets o = 0.
 *   A sequence without queries (n = 0) is not read.
 *
 * Layouts (row-major; bf16 values as their 16-bit patterns). The tokens of
 * the B sequences are packed end to end: sequence b owns tokens offsets[b] ..
 * offsets[b+1]-1 of the call.
 *   k_codes, v_codes    uint8_t  [B][Hkv][L_max][D]
 *   k_scales, v_scales  float    [B][Hkv][ceil(L_max / block)]
 *   k_new, v_new        uint16_t [T][Hkv][D], kv_stride elements from token to token
 *   q                   uint16_t [T][Hq][D], q_stride elements from token to token
 *   o                   uint16_t [T][Hq][D] packed
 *   k_out, v_out        uint16_t [T][Hkv][D] packed
 *   offsets             int32_t  [B+1]  0 = offsets[0] <= ... <= offsets[B] = T
 *   starts              int32_t  [B]    starts[b] >= 0, starts[b] + n <= L_max
 *   lens                int32_t  [B]    0 <= lens[b] <= L_max
 *
 * Ownership, streams and errors as in moe.h: device pointers owned by the
 * caller, host shape pointer, no allocation, no state between calls, no host
 * synchronisation, all work on `stream`. Argument errors are returned
 * synchronously. offsets, starts and lens are read on the device: when any of
 * them breaks the rules above, MOE_ERR_INVALID_ARG is written to the status
 * word and nothing else is written. Outputs must not overlap inputs. Results
 * are bit-identical from run to run.
 */
#ifndef BGMOE_KV8_H
#define BGMOE_KV8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_kv8_format {
  MOE_KV8_INT8 = 0,
  MOE_KV8_E4M3 = 1
} moe_kv8_format;

/* Shape of one call. Supported: 1 <= B <= 4096; 0 <= T <= 2^24; 1 <= Hkv <=
 * 4096, B * Hkv <= 65536, T * Hkv <= 2^30; Hq a multiple of Hkv with Hq / Hkv
 * <= 64; D in {64, 128, 256}; 1 <= L_max <= 2^26; block in {16, 32, 64}.
 * Strides: 0 for packed tokens, or a multiple of 8 elements of at least one
 * token's (Hq D, Hkv D).
 * Write and read do not use Hq and q_stride, attention not kv_stride; they
 * are checked all the same. */
typedef struct moe_kv8_shape {
  int32_t B;         /* sequences */
  int32_t T;         /* tokens of all sequences in this call (new, read or querying) */
  int32_t Hq;        /* query heads */
  int32_t Hkv;       /* key/value heads */
  int32_t D;         /* head size */
  int32_t L_max;     /* cache rows per (sequence, KV head) */
  int32_t block;     /* positions per scale */
  int32_t format;    /* moe_kv8_format */
  int32_t q_stride;  /* elements between the tokens of q (0: Hq * D) */
  int32_t kv_stride; /* elements between the tokens of k_new and v_new (0: Hkv * D) */
} moe_kv8_shape;

/* A cache's device arrays. */
typedef struct moe_kv8_cache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
} moe_kv8_cache;

/* Quantises T new tokens into the cache. k_new, v_new and the codes must be
 * 16-byte aligned, the rest 4-byte aligned. `status`: an int32 device word
 * that the caller zeroed, or NULL. T == 0 is a no-op. */
moe_status moe_kv8_write(const moe_kv8_shape* shape, const void* k_new, const void* v_new, const int32_t* offsets,
                         const int32_t* starts, const moe_kv8_cache* cache, int32_t* status, void* stream);

/* Reads T positions back as bf16. Alignments and status as moe_kv8_write
 * (k_out and v_out 16-byte aligned). */
moe_status moe_kv8_read(const moe_kv8_shape* shape, const moe_kv8_cache* cache, const int32_t* offsets,
                        const int32_t* starts, void* k_out, void* v_out, int32_t* status, void* stream);

/* Bytes of device workspace moe_kv8_attn needs for `shape`, or with fewer tokens
 * (T): a workspace for the largest T serves all steps of one cache. */
moe_status moe_kv8_workspace_bytes(const moe_kv8_shape* shape, size_t* bytes);

/* Causal attention of T query tokens over the cache (the formula above). q,
 * o and the codes must be 16-byte aligned, the workspace 256-byte aligned
 * with ws_bytes >= moe_kv8_workspace_bytes(); its contents need no
 * initialisation, and calls that may overlap on the GPU need one each. `scale`
 * must be finite and > 0 (1/sqrt(D) is the usual value). The int32 at the
 * start of the workspace is the call's status word (read it with
 * moe_status_read): MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_DEVICE_TIMEOUT (a
 * bounded wait ran out; o is not valid). T == 0 writes the status word only.
 * The kernels are chosen by the tokens per sequence on average: a batch of
 * single tokens and a long chunk is quicker as two calls, the chunk's on the
 * cache rows of its sequences alone (any range of B is a cache).
 *
 * Numerics: q goes to fp16 with its row's largest magnitude in [1, 2) (values
 * 2^-14 below that lose bits), codes are exact; the weights, softmax times V's
 * scale, go to fp16 with the row's running maximum at 2^7 to 2^15; products,
 * softmax and sums are fp32, and o is rounded once to bf16. So o is within
 *   2^-8 |o| + 2.1 * 2^-11 sum_j p_j |V_j|
 *            + 2^-32 max_j (p_j s_v(j)) sum_j |c_j|
 * of the formula (c_j: V's code, s_v(j): its scale, 2^-60 for zeros; the last
 * term is for weights 2^-21 and more below the largest, where fp16's steps no
 * longer shrink), and of what errors of the scores do to p: q's rounding, and
 * fp32's of a sum of D products and of adding log2 s_v(j), up to 2^-22 of the
 * score's size (positions whose scores are nearer to one another than that
 * share their weight in some way). V's scales may lie any distance apart. Where
 * scale * log2(e) * max|q| * k_scale, a score or an output passes fp32's range,
 * the row has infinities or NaN.
 */
moe_status moe_kv8_attn(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache, const int32_t* offsets,
                        const int32_t* lens, float scale, void* o, void* workspace, size_t ws_bytes, void* stream);

/* Test hook for the bounded waits (failure detection): moe_kv8_attn in which
 * grid block `stalled_block` (0-based, below the grid of one block per SM; a
 * block past the grid or without work changes nothing) never brings its
 * operands, so that the waits of its other warps run out after `timeout_ns`
 * (0 < timeout_ns <= 1 s), as do those of a block that works with it. The
 * call's status word then reads MOE_ERR_DEVICE_TIMEOUT, no block exits with a
 * copy or a product in flight, o is not valid, and the context stays usable.
 * INVALID_ARG for a negative block or a timeout out of range; the other
 * checks are moe_kv8_attn's. */
moe_status moe_kv8_attn_test_stall(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache,
                                   const int32_t* offsets, const int32_t* lens, float scale, void* o, void* workspace,
                                   size_t ws_bytes, int32_t stalled_block, int64_t timeout_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BGMOE_KV8_H */
