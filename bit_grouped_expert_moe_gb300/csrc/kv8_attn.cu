// Causal grouped-query attention over the 8-bit KV cache (include/kv8.h):
// argument checks and the choice between its two kinds of kernels.
#include "kernels.h"
#include "kv8_attn.h"

namespace bgmoe {
namespace kv8 {

int sm_count() {
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (sms[dev] == 0 && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms[dev] = 0;
  return sms[dev];
}

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Which kernels serve a call: the split-context ones read the cache once per 8
// to 32 rows (query heads of a KV head x tokens), the tiles once per 128 or 256
// but with a longer chain in front. So a call is the former's with up to 36
// rows per sequence and KV head, or somewhat more where few of those pairs
// keep the GPU's blocks from filling up. Measured, split / tiles in us, INT8, n
// tokens of each of B sequences over L positions:
//   16 heads / 2 x 256, B = 1, L = 32,768:   n = 12 49.0 / 55.8, n = 16 61.9 / 56.6
//                       B = 1, L = 2048:     n = 64 29.1 / 32.3
//                       B = 16, L = 4096:    n = 4 42.6 / 47.2, n = 8 73.8 / 47.8
//                       B = 16, L = 512:     n = 4 18.9 / 23.2, n = 8 28.6 / 23.7
//   16 heads / 4 x 128, B = 1, L = 32,768:   n = 24 39.5 / 43.7, n = 32 48.5 / 44.6
//                       B = 16, L = 4096:    n = 12 59.4 / 60.7, n = 24 87.9 / 62.4
//                       B = 16, L = 512:     n = 8 19.2 / 22.2, n = 12 25.6 / 22.4
//   8 heads / 8 x 128,  B = 1, L = 32,768:   n = 64 50.0 / 61.1
//                       B = 16, L = 512:     n = 32 28.1 / 28.9, n = 64 45.7 / 29.2
//   4 heads / 1 x 64,   B = 16, L = 4096:    n = 12 16.9 / 19.6, n = 24 25.0 / 20.7
//   40 heads / 8 x 128, B = 16, L = 4096:    n = 4 58.4 / 110, n = 8 105 / 103
// The host knows the tokens of the batch, not each sequence's, so one long chunk
// among many single tokens goes with them, at either side of the rule to its or
// their cost (16 heads / 2 x 256, one call / the two alone, in us):
//   63 tokens over 4000 each and 100 over 20,000:      274 (split)  / 58 + 58
//   63 tokens over 4000 each and 1000 over 20,000:     358 (tiles)  / 58 + 251
//   255 tokens over 1000 each and 800 over 32,768:    2781 (split)  / 123 + 298
bool few(const moe_kv8_shape& s) { return (long long)s.T * s.Hq <= 36ll * s.B * s.Hkv + 192; }

// For up to s.T tokens: what the tiles need does not grow with T, while the split
// kernels' partial states do, so fewer tokens may need more. Theirs grow while
// the rows per tile stay the same; split_steps are the T at which those change.
size_t workspace_bytes(const moe_kv8_shape& s) {
  if (s.T == 0) return 256;
  size_t most = few(s) ? 0 : tiles_workspace_bytes(s);
  const long long last = (36ll * s.B * s.Hkv + 192) / s.Hq;  // the most tokens that few() takes
  long long T[3] = {last};
  split_steps(s, T + 1);
  for (const long long t : T) {
    moe_kv8_shape fewer = s;
    fewer.T = (int32_t)(t < s.T ? t : s.T);
    if (fewer.T > 0 && few(fewer)) {
      const size_t n = split_workspace_bytes(fewer);
      most = n > most ? n : most;
    }
  }
  return most;
}

moe_status attn(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache, const int32_t* offsets,
                const int32_t* lens, float scale, void* o, void* workspace, size_t ws_bytes, void* stream,
                int stalled = -1, long long timeout_ns = kTimeoutNs) {
  if (!shape) return MOE_ERR_INVALID_ARG;
  const moe_kv8_shape s = *shape;
  if (!shape_ok(s)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!cache_ok(cache) || !aligned(offsets, 4) || !aligned(lens, 4) || !aligned(q, 16) || !aligned(o, 16) ||
      !workspace || !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < workspace_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.T == 0) {
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), st);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "status clear");
  }
  if (!q || !offsets || !lens || !o) return MOE_ERR_INVALID_ARG;
  const AttnArgs a{static_cast<const uint16_t*>(q), cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales,
                   offsets, lens, static_cast<uint16_t*>(o), workspace, s.B, s.T, s.Hq, s.Hkv, s.D, s.L_max,
                   (s.L_max + s.block - 1) / s.block, s.block, s.format == MOE_KV8_E4M3,
                   s.q_stride ? s.q_stride : s.Hq * s.D, scale * kLog2e, stalled, timeout_ns};
  return few(s) ? launch_split(a, st) : launch_tiles(a, st);
}

}  // namespace
}  // namespace kv8
}  // namespace bgmoe

extern "C" {

moe_status moe_kv8_workspace_bytes(const moe_kv8_shape* shape, size_t* bytes) {
  if (!shape || !bytes) return MOE_ERR_INVALID_ARG;
  if (!bgmoe::kv8::shape_ok(*shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = bgmoe::kv8::workspace_bytes(*shape);
  return MOE_OK;
}

moe_status moe_kv8_attn(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache, const int32_t* offsets,
                        const int32_t* lens, float scale, void* o, void* workspace, size_t ws_bytes, void* stream) {
  return bgmoe::kv8::attn(shape, q, cache, offsets, lens, scale, o, workspace, ws_bytes, stream);
}

moe_status moe_kv8_attn_test_stall(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache,
                                   const int32_t* offsets, const int32_t* lens, float scale, void* o, void* workspace,
                                   size_t ws_bytes, int32_t stalled_block, int64_t timeout_ns, void* stream) {
  if (stalled_block < 0 || timeout_ns <= 0 || timeout_ns > bgmoe::kv8::kTimeoutNs) return MOE_ERR_INVALID_ARG;
  return bgmoe::kv8::attn(shape, q, cache, offsets, lens, scale, o, workspace, ws_bytes, stream, stalled_block,
                          timeout_ns);
}

}  // extern "C"
