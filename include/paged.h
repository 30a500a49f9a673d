/*
 * bit_grouped_expert_moe_gb300 — C ABI of a paged bf16 KV cache for NVIDIA
 * GB300 (sm_103a): new tokens appended with norm and rotation on the way,
 * grouped-query attention over it (one token per sequence, trees of drafted
 * tokens, chunks and whole prompts), and the accepted path of a tree kept.
 *
 * The cache is two pools of pages and a table. Position p of sequence b is row
 * p % page of page tables[b][p / page] of either pool:
 *   k_pages, v_pages  uint16_t [n_pages][Hkv][page][D]  (bf16)
 *   tables            int32_t  [B][max_pages]
 * Entries of the table past a sequence's positions are not read, and rows past
 * them may hold anything. Sequences may share pages that no call writes.
 *
 * The tokens of the B sequences are packed end to end: sequence b owns tokens
 * offsets[b] .. offsets[b+1]-1 of the call.
 *
 * Append: token i of sequence b goes to position starts[b] + i: its value as
 *   it is, its key normed and rotated (rope.h) by the position positions[t],
 *   or starts[b] + i without `positions` (a draft in a tree has the position
 *   of its depth, not of its place). Its query, if given, is normed and
 *   rotated into q_out alongside.
 *
 * Attention: the queries of sequence b are its last n = offsets[b+1] -
 *   offsets[b] positions, lens[b] in all:
 *     o[i,h,:] = sum_j softmax_j(scale * q[i,h,:] . K[b,g,j,:]) V[b,g,j,:],
 *     g = h / (Hq / Hkv),
 *   over the positions j >= 0 that query i sees: j <= lens[b] - n + i (its own
 *   key included), and with a tree those of the new positions lens[b] - n + d
 *   only whose draft d has its bit in the query's words: bit d % 64 of
 *   tree[t][d / 64] (a draft's ancestors and itself; bits of later drafts
 *   count for nothing). A query that sees no position gets o = 0. A
 *   sequence without queries is not read. What a query does not see has no
 *   part in its result, whatever it holds, infinities and NaN included.
 *
 * Keep: for sequence b the rows of drafts path[b][0] < path[b][1] < ... <
 *   path[b][kept[b]-1], at positions starts[b] + path[b][k], move to positions
 *   starts[b] + k: the accepted path follows the context without gaps.
 *   lens_out[b] = starts[b] + kept[b].
 *
 * Layouts (row-major; bf16 values as their 16-bit patterns)
 *   q            uint16_t [T][Hq][D], q_stride elements from token to token
 *   k_new, v_new uint16_t [T][Hkv][D], kv_stride elements from token to token
 *   q_out, o     uint16_t [T][Hq][D] packed
 *   offsets      int32_t  [B+1]  0 = offsets[0] <= ... <= offsets[B] = T
 *   starts       int32_t  [B]    starts[b] >= 0, starts[b] + n <= max_pages * page
 *   lens         int32_t  [B]    0 <= lens[b] <= max_pages * page
 *   positions    int32_t  [T]
 *   tree         uint64_t [T][tree_words]
 *   path         int32_t  [B][path_stride], kept int32_t [B]
 *
 * Ownership, streams and errors as in moe.h: device pointers owned by the
 * caller, host shape pointer, no allocation, no state between calls, no host
 * synchronisation, all work on `stream`. Argument errors are returned
 * synchronously. Tables of indices (offsets, starts, lens, positions, tables,
 * kept, path) are read on the device, so a captured call can be replayed with
 * others; where they break the rules above, MOE_ERR_INVALID_ARG is written to
 * the status word and no access leaves the arrays (each call says what is
 * written then). Outputs must not overlap inputs. Results are bit-identical
 * from run to run.
 */
#ifndef BGMOE_PAGED_H
#define BGMOE_PAGED_H

#include "rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of one call. Supported: 1 <= B <= 4096; 0 <= T <= 2^24; 1 <= Hkv <=
 * 4096, B * Hkv <= 65536, T * Hkv <= 2^30; Hq a multiple of Hkv with Hq / Hkv
 * <= 64; D in {64, 128, 256}; page in {16, 32, 64, 128, 256}; 1 <= n_pages,
 * n_pages * Hkv <= 2^31 - 1; 1 <= max_pages, max_pages * page <= 2^26;
 * 0 <= tree_words <= 8. Strides: 0 for packed tokens, or a multiple of 8
 * elements of at least one token's (Hq D, Hkv D).
 * Append does not use tree_words, attention not kv_stride, keep neither T, Hq,
 * nor strides; all are checked all the same. */
typedef struct moe_paged_shape {
  int32_t B;          /* sequences */
  int32_t T;          /* tokens of all sequences in this call (new or querying) */
  int32_t Hq;         /* query heads */
  int32_t Hkv;        /* key/value heads */
  int32_t D;          /* head size */
  int32_t page;       /* positions per page */
  int32_t n_pages;    /* pages of the pools */
  int32_t max_pages;  /* entries of a sequence's row of the table */
  int32_t tree_words; /* 64-bit words of a draft's mask, 0: causal */
  int32_t q_stride;   /* elements between the tokens of q (0: Hq * D) */
  int32_t kv_stride;  /* elements between the tokens of k_new and v_new (0: Hkv * D) */
} moe_paged_shape;

/* The pools and the table. */
typedef struct moe_paged_cache {
  void* k_pages;
  void* v_pages;
  const int32_t* tables;
} moe_paged_cache;

/* Appends T new tokens. `spec` as in moe_rope, or NULL: keys and queries as
 * they are. q and q_out: both or neither; q_out may be q if its tokens are
 * packed. positions may be NULL. q, k_new, v_new, q_out and the pools must be
 * 16-byte aligned, the rest 4-byte aligned. `status`: an int32 device word that the caller zeroed,
 * or NULL. A token whose sequence, position or page breaks the rules is not
 * written (nor its query). Two tokens for one row of a page leave either's
 * heads, of each head one token's.
 * T == 0 is a no-op. */
moe_status moe_paged_append(const moe_paged_shape* shape, const moe_rope_spec* spec, const void* q, const void* k_new,
                            const void* v_new, const int32_t* offsets, const int32_t* starts, const int32_t* positions,
                            const moe_paged_cache* cache, void* q_out, int32_t* status, void* stream);

/* Bytes of device workspace moe_paged_attn needs for `shape`, whatever its T. */
moe_status moe_paged_workspace_bytes(const moe_paged_shape* shape, size_t* bytes);

/* Attention of T query tokens over the cache (the formula above). `tree` is
 * NULL if and only if tree_words is 0 (8-byte aligned). q, o and the pools
 * must be 16-byte aligned, the workspace 256-byte aligned with ws_bytes >=
 * moe_paged_workspace_bytes(); its contents need no initialisation, and calls
 * that may overlap on the GPU need one each. `scale` must be > 0 and below
 * 2.35e38, so that scale log2(e) is finite in fp32 (1/sqrt(D) is the usual
 * value). The int32 at the start of the workspace is
 * the call's status word (read it with moe_status_read): MOE_OK,
 * MOE_ERR_INVALID_ARG or MOE_ERR_DEVICE_TIMEOUT (a bounded wait ran out; o is
 * not valid). Where offsets or lens break the rules, or a sequence has more
 * than 64 * tree_words drafts, nothing else is written; where a page that a
 * sequence's positions need is not in the pools, o is not valid.
 * T == 0 writes the status word only.
 *
 * Numerics: scores from exact products of bf16, summed in fp32; weights
 * relative to a running maximum that the row's largest score passes by a
 * factor of 2^8 at most, their sum in fp32, each rounded to bf16 for the
 * product with V; o is rounded once to bf16. So o is within
 *   2^-8 |o| + (2^-8 + 2^-15) sum_j p_j |V_j|
 * of the formula (2^-15: the exponents, whatever the size of the scores), and of
 * what fp32's errors of the scores and the sums do to p. In calls
 * with T * Hq <= 16 * B * Hkv the running maximum is the largest score so far,
 * and the sum is without the position that has it (its weight is 1, to 2^-17).
 * A query that sees a value of V which is infinite or NaN has NaN or infinities
 * in its output, and is NaN throughout where that position is not seen by all
 * queries that share its tile. One that sees a score of infinity or NaN, or no
 * score but minus infinity, is NaN; minus infinity beside other scores weighs
 * nothing. (Scores are formed in fp32, before the scale: from 2^126 on they may
 * count as infinite.)
 */
moe_status moe_paged_attn(const moe_paged_shape* shape, const void* q, const moe_paged_cache* cache,
                          const int32_t* offsets, const int32_t* lens, const uint64_t* tree, float scale, void* o,
                          void* workspace, size_t ws_bytes, void* stream);

/* Test hook for the bounded waits (failure detection): moe_paged_attn in which
 * grid block `stalled_block` (0-based; a block past the grid or without work
 * changes nothing) never brings its keys and values, so that the waits of its
 * other warps run out after `timeout_ns` (0 < timeout_ns <= 1 s), as do those
 * of a block that works with it. The call's status word then reads
 * MOE_ERR_DEVICE_TIMEOUT, no block exits with a copy or a product in flight, o
 * is not valid, and the context stays usable. INVALID_ARG for a negative block
 * or a timeout out of range; the other checks are moe_paged_attn's. */
moe_status moe_paged_attn_test_stall(const moe_paged_shape* shape, const void* q, const moe_paged_cache* cache,
                                     const int32_t* offsets, const int32_t* lens, const uint64_t* tree, float scale,
                                     void* o, void* workspace, size_t ws_bytes, int32_t stalled_block,
                                     int64_t timeout_ns, void* stream);

/* Keeps the accepted drafts (above). 0 <= kept[b] <= path_stride <= 512, and
 * path[b] is read up to kept[b]. The pools must be 16-byte aligned, the rest
 * 4-byte aligned; lens_out and status may be NULL.
 * A sequence whose entries break the rules is left as it was. */
moe_status moe_paged_keep(const moe_paged_shape* shape, const moe_paged_cache* cache, const int32_t* starts,
                          const int32_t* kept, const int32_t* path, int32_t path_stride, int32_t* lens_out,
                          int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BGMOE_PAGED_H */
