// Causal grouped-query attention over the 8-bit KV cache (include/kv8.h), sm_103a.
//
// One warp per (query token, query head): the lanes share the head dimension
// and walk the visible positions with the running maximum and sum of a
// softmax, so the scores are never stored.
#include "kernels.h"
#include "kv8_attn.h"

#include <type_traits>

namespace bgmoe {
namespace kv8 {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) kv8_rows_kernel(const AttnArgs p) {
  constexpr int kPer = D / 32 < 4 ? 4 : D / 32;  // values per lane
  constexpr int kLanes = D / kPer;               // lanes that hold some
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(row / p.Hq), h = (int)(row % p.Hq);
  int b = 0, i = 0, n = 0, len = 0;
  bool bad = false;
  for (int base = 0; base < p.B; base += 32) {
    const int bb = base + lane;
    int lo = 0, hi = 0, L = 0;
    if (bb < p.B) {
      lo = __ldg(p.offsets + bb);
      hi = __ldg(p.offsets + bb + 1);
      L = __ldg(p.lens + bb);
      bad |= offsets_bad(lo, hi, bb, p.B, p.T) || L < 0 || L > p.L_max;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, bb < p.B && t >= lo && t < hi);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b = base + l;
      i = t - __shfl_sync(0xffffffffu, lo, l);
      n = __shfl_sync(0xffffffffu, hi - lo, l);
      len = __shfl_sync(0xffffffffu, L, l);
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (row == 0 && lane == 0) *static_cast<int32_t*>(p.workspace) = bad ? (int32_t)MOE_ERR_INVALID_ARG : 0;
  if (bad || t >= p.T) return;
  const int g = h / (p.Hq / p.Hkv);
  const size_t pair = (size_t)b * p.Hkv + g;
  const int seen = len - n + i + 1;  // visible positions (<= len)
  const int d0 = (lane % kLanes) * kPer;
  float q[kPer], acc[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    q[j] = lane < kLanes ? bf16_bits_to_f32(p.q[(size_t)t * p.q_stride + (size_t)h * D + d0 + j]) : 0.f;
    acc[j] = 0.f;
  }
  float m = -1e30f, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const size_t at = (pair * p.L_max + j) * D + d0;
    const size_t sat = pair * p.nblk + j / p.block;
    float s = 0.f, kf[4], vf[kPer];
#pragma unroll
    for (int c = 0; c < kPer; c += 4) {
      decode4<kE4m3>(*reinterpret_cast<const uint32_t*>(p.k + at + c), kf);
      decode4<kE4m3>(*reinterpret_cast<const uint32_t*>(p.v + at + c), *reinterpret_cast<float(*)[4]>(&vf[c]));
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(q[c + e], kf[e], s);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.ks[sat] * p.scale_log2;
    const float nm = fmaxf(m, s), f = exp2f(m - nm), w = exp2f(s - nm);
    m = nm;
    l = l * f + w;
    const float wv = w * p.vs[sat];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = fmaf(acc[c], f, wv * vf[c]);
  }
  if (lane < kLanes) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const __nv_bfloat16 r = __float2bfloat16_rn(seen > 0 ? acc[j] / l : 0.f);
      p.o[((size_t)t * p.Hq + h) * D + d0 + j] = __bfloat16_as_ushort(r);
    }
  }
}

namespace {

// Few query tokens per sequence: the split-context kernels; more: one warp per row.
bool few(const moe_kv8_shape& s) { return s.T <= 8 * s.B; }

size_t workspace_bytes(const moe_kv8_shape& s) { return few(s) ? split_workspace_bytes(s) : 256; }

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
  int32_t* status = static_cast<int32_t*>(workspace);
  if (s.T == 0) {
    const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), st);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "status clear");
  }
  if (!q || !offsets || !lens || !o) return MOE_ERR_INVALID_ARG;
  AttnArgs p{static_cast<const uint16_t*>(q), cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales, offsets,
             lens, static_cast<uint16_t*>(o), workspace, s.B, s.T, s.Hq, s.Hkv, s.D, s.L_max,
             (s.L_max + s.block - 1) / s.block, s.block, s.format == MOE_KV8_E4M3,
             s.q_stride ? s.q_stride : s.Hq * s.D, scale * kLog2e};
  if (few(s)) return launch_split(p, st);
  const unsigned grid = (unsigned)(((long long)s.T * s.Hq + kWarps - 1) / kWarps);
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (s.format == MOE_KV8_E4M3) kv8_rows_kernel<D, true><<<grid, kWarps * 32, 0, st>>>(p);
    else kv8_rows_kernel<D, false><<<grid, kWarps * 32, 0, st>>>(p);
  };
  if (s.D == 64) go(std::integral_constant<int, 64>{});
  else if (s.D == 128) go(std::integral_constant<int, 128>{});
  else go(std::integral_constant<int, 256>{});
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attention launch");
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
