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
// keep the GPU's blocks from filling up. (The host knows the tokens of the
// batch, not each sequence's.) Measured, split / tiles in us, INT8, n tokens of
// each of B sequences over L positions:
//   16 heads / 2 x 256, B = 1, L = 32,768:   n = 12 48.5 / 55.9, n = 16 60.8 / 57.3
//                       B = 1, L = 2048:     n = 64 28.4 / 32.8
//                       B = 16, L = 4096:    n = 4 41.9 / 47.6, n = 8 73.0 / 48.0
//                       B = 16, L = 512:     n = 4 18.5 / 23.2, n = 8 27.6 / 23.7
//   16 heads / 4 x 128, B = 1, L = 32,768:   n = 24 38.2 / 43.3, n = 32 47.0 / 44.3
//                       B = 16, L = 4096:    n = 12 57.4 / 59.2, n = 24 84.6 / 61.3
//                       B = 16, L = 512:     n = 8 18.4 / 21.9, n = 12 24.2 / 22.1
//   8 heads / 8 x 128,  B = 1, L = 32,768:   n = 64 48.7 / 60.5
//                       B = 16, L = 512:     n = 32 26.5 / 28.6, n = 64 43.0 / 28.8
//   4 heads / 1 x 64,   B = 16, L = 4096:    n = 12 16.5 / 19.1, n = 24 24.5 / 20.3
//   40 heads / 8 x 128, B = 16, L = 4096:    n = 4 57.2 / 107, n = 8 102 / 100
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
