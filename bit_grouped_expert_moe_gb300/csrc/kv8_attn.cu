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

// Few query tokens per sequence: the split-context kernels; more: the tiles.
bool few(const moe_kv8_shape& s) { return s.T <= 8 * s.B; }

size_t workspace_bytes(const moe_kv8_shape& s) {
  return s.T == 0 ? 256 : few(s) ? split_workspace_bytes(s) : tiles_workspace_bytes(s);
}

moe_status attn(const moe_kv8_shape* shape, const void* q, const moe_kv8_cache* cache, const int32_t* offsets,
                const int32_t* lens, float scale, void* o, void* workspace, size_t ws_bytes, void* stream) {
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
                   s.q_stride ? s.q_stride : s.Hq * s.D, scale * kLog2e};
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

}  // extern "C"
