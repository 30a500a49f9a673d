// Writing into and reading back from the 8-bit KV cache (include/kv8.h), sm_103a.
//
// Both move bytes and compute almost nothing: a value costs one multiply and
// one conversion, so they are bound by memory, and at a decode step's sizes
// by the latency of one dependent chain (tables, values, scale, codes).
#include "kernels.h"
#include "kv8.cuh"

#include <type_traits>

namespace bgmoe {
namespace kv8 {

constexpr int kThreads = 256;
constexpr int kReadTokens = 64;  // packed tokens per block of the read kernel

struct CacheArgs {
  uint8_t* codes[2];    // K, V
  float* scales[2];
  const uint16_t* x[2]; // write: new tokens
  uint16_t* out[2];     // read: bf16 values
  const int32_t* offsets;
  const int32_t* starts;
  int32_t* status;
  int B, T, Hkv, L_max, nblk;
  int stride;           // elements from token to token of x
};

__device__ __forceinline__ void flag(int32_t* status, int32_t what) {
  if (status) atomicCAS(status, 0, what);
}

// Every thread block checks the whole table (a load or two per thread for
// the usual batch): a call with a bad entry writes nothing anywhere. hit(b,
// lo, hi, start) runs for every sequence.
template <typename Hit>
__device__ __forceinline__ bool tables_bad(const CacheArgs& p, Hit hit) {
  bool bad = false;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int lo = __ldg(p.offsets + b), hi = __ldg(p.offsets + b + 1), start = __ldg(p.starts + b);
    if (offsets_bad(lo, hi, b, p.B, p.T) || range_bad(start, hi - lo, p.L_max)) bad = true;
    else hit(b, lo, hi, start);
  }
  return __syncthreads_or(bad) != 0;
}

// One thread block per (touched cache block, KV head, K or V). Sequence b's
// touched blocks are units floor(offsets[b] / kBlock) + 2 b + 0, 1, ...: n
// tokens touch at most floor(n / kBlock) + 2 blocks, which is what the next
// sequence's first unit leaves room for, so no prefix sum is needed and the
// grid is floor(T / kBlock) + 2 B (units that touch nothing return).
//
// The block's new values stay in registers between the maximum and the codes
// (64 x 256 bf16 over 256 threads: 8 16-byte pieces each), so they are read
// once, all loads in flight together.
template <int D, int kBlock, bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(const CacheArgs p) {
  constexpr int kPieces = kBlock * D / 8;             // 16-byte pieces (8 values) of a full block
  constexpr int kPer = (kPieces + kThreads - 1) / kThreads;
  __shared__ int s_b, s_lo, s_n, s_start;
  __shared__ uint32_t s_max[kThreads / 32];
  const int unit = blockIdx.x, g = blockIdx.y, kv = blockIdx.z;
  if (threadIdx.x == 0) s_b = -1;
  __syncthreads();
  const bool bad = tables_bad(p, [&](int b, int lo, int hi, int start) {
    const int u0 = lo / kBlock + 2 * b, u1 = hi / kBlock + 2 * (b + 1);
    if (unit >= u0 && unit < u1) {
      s_b = b;
      s_lo = lo;
      s_n = hi - lo;
      s_start = start;
    }
  });
  if (bad) {
    if (threadIdx.x == 0) flag(p.status, (int32_t)MOE_ERR_INVALID_ARG);
    return;
  }
  const int b = s_b;
  if (b < 0) return;
  const int n = s_n, start = s_start;
  const int blk = start / kBlock + (unit - (s_lo / kBlock + 2 * b));
  const int base = blk * kBlock;                       // the cache block's first position
  const int p0 = max(start, base), p1 = min(start + n, base + kBlock);  // its new positions
  if (n == 0 || p0 >= p1) return;
  const size_t pair = (size_t)b * p.Hkv + g;
  uint8_t* codes = p.codes[kv] + (pair * p.L_max + base) * D;
  float* scale = p.scales[kv] + pair * p.nblk + blk;
  const float s_old = p0 > base ? *scale : 0.f;
  const uint16_t* x = p.x[kv] + (size_t)g * D;
  const int r0 = p0 - base, r1 = p1 - base;            // rows of the block
  const int t0 = s_lo + (p0 - start);                  // the packed token of row r0

  uint4 v[kPer];
  uint32_t mx = 0;  // largest magnitude bits, two bf16 side by side
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = threadIdx.x + i * kThreads;      // piece of the new rows, from row r0
    const int row = piece / (D / 8), c = piece % (D / 8);
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < r1 - r0) v[i] = ldg_nc_v4(x + (size_t)(t0 + row) * p.stride + c * 8);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, w[j] & 0x7FFF7FFFu);
  }
  auto block_max = [&](uint32_t m2) -> uint32_t {      // over both halves and all threads
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, s_max[w]);
    return m;
  };
  uint32_t m = block_max(mx);
  if (m >= 0x7F80u) {  // an infinity or a NaN: the maximum again over finite values, then replace them
    if (threadIdx.x == 0) flag(p.status, (int32_t)MOE_ERR_RANGE);
    __syncthreads();   // s_max is read above
    mx = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) mx = max(mx & 0xFFFFu, lo) | (mx & 0xFFFF0000u);
        if (hi < 0x7F80u) mx = max(mx >> 16, hi) << 16 | (mx & 0xFFFFu);
      }
    }
    m = block_max(mx);
    auto finite = [&](uint32_t h) -> uint32_t {        // one bf16
      const uint32_t a = h & 0x7FFFu;
      return a < 0x7F80u ? h : a == 0x7F80u ? (h & 0x8000u) | m : 0u;
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i].x = finite(v[i].x & 0xFFFFu) | finite(v[i].x >> 16) << 16;
      v[i].y = finite(v[i].y & 0xFFFFu) | finite(v[i].y >> 16) << 16;
      v[i].z = finite(v[i].z & 0xFFFFu) | finite(v[i].z >> 16) << 16;
      v[i].w = finite(v[i].w & 0xFFFFu) | finite(v[i].w >> 16) << 16;
    }
  }
  const float s_new = fmaxf(s_old, scale_of<kE4m3>(__uint_as_float(m << 16)));
  const float inv = inverse_scale(s_new);
  if (p0 > base && s_new > s_old) {  // the block's earlier codes, to the larger scale
    for (int piece = threadIdx.x; piece < r0 * (D / 4); piece += kThreads) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes) + piece;
      float f[4];
      decode4<kE4m3>(*w, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = f[j] * s_old * inv;
        if (!kE4m3) f[j] = fmaxf(f[j], -127.f);  // a byte of code -128 (no write stores one)
      }
      *w = encode4<kE4m3>(f[0], f[1], f[2], f[3]);
    }
  }
  if (threadIdx.x == 0 && (p0 == base || s_new != s_old)) *scale = s_new;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    const int row = piece / (D / 8), c = piece % (D / 8);
    if (row >= r1 - r0) continue;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float f0 = __uint_as_float(w[2 * j] << 16), f1 = __uint_as_float(w[2 * j] & 0xFFFF0000u);
      const float f2 = __uint_as_float(w[2 * j + 1] << 16), f3 = __uint_as_float(w[2 * j + 1] & 0xFFFF0000u);
      o[j] = encode4<kE4m3>(f0 * inv, f1 * inv, f2 * inv, f3 * inv);
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(r0 + row) * D + c * 8) = make_uint2(o[0], o[1]);
  }
}

// One thread block per (64 packed tokens, KV head, K or V): the sequence of
// every token is found first, then each thread turns 8-byte pieces of codes
// into 16-byte pieces of bf16, so a warp reads and writes whole lines.
template <int D, int kBlock, bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const CacheArgs p) {
  __shared__ int s_row[kReadTokens], s_seq[kReadTokens];  // cache position and sequence of each token
  const int t0 = blockIdx.x * kReadTokens, g = blockIdx.y, kv = blockIdx.z;
  const int nt = min(kReadTokens, p.T - t0);
  const bool bad = tables_bad(p, [&](int b, int lo, int hi, int start) {
    const int a = max(lo, t0), z = min(hi, t0 + nt);
    for (int t = a; t < z; ++t) {
      s_row[t - t0] = start + (t - lo);
      s_seq[t - t0] = b;
    }
  });
  if (bad) {
    if (threadIdx.x == 0) flag(p.status, (int32_t)MOE_ERR_INVALID_ARG);
    return;
  }
  constexpr int kRow = D / 8;                           // pieces per token
  constexpr int kPer = kReadTokens * kRow / kThreads;
  const uint8_t* codes = p.codes[kv];
  const float* scales = p.scales[kv];
  uint2 w[kPer];
  float s[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = threadIdx.x + i * kThreads, t = piece / kRow, c = piece % kRow;
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (t < nt) {
      const size_t pair = (size_t)s_seq[t] * p.Hkv + g;
      const int pos = s_row[t];
      w[i] = __ldcs(reinterpret_cast<const uint2*>(codes + (pair * p.L_max + pos) * D + c * 8));
      s[i] = __ldg(scales + pair * p.nblk + pos / kBlock);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = threadIdx.x + i * kThreads, t = piece / kRow, c = piece % kRow;
    if (t >= nt) continue;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float f[4];
      decode4<kE4m3>(j ? w[i].y : w[i].x, f);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0] * s[i], f[1] * s[i]);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(f[2] * s[i], f[3] * s[i]);
      o[2 * j] = *reinterpret_cast<const uint32_t*>(&lo);
      o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
    __stcs(reinterpret_cast<uint4*>(p.out[kv] + ((size_t)(t0 + t) * p.Hkv + g) * D + c * 8),
           make_uint4(o[0], o[1], o[2], o[3]));
  }
}

// ================================================================= host ===

bool shape_ok(const moe_kv8_shape& s) {
  if (s.B < 1 || s.B > 4096 || s.T < 0 || s.T > (1 << 24)) return false;
  if (s.Hkv < 1 || s.Hkv > 4096 || s.Hq < 1 || s.Hq % s.Hkv != 0) return false;
  if (s.Hq / s.Hkv > 64 || (long long)s.B * s.Hkv > 65536) return false;
  if (s.D != 64 && s.D != 128 && s.D != 256) return false;
  if (s.L_max < 1 || s.L_max > (1 << 26) || (s.block != 16 && s.block != 32 && s.block != 64)) return false;
  if (s.format != MOE_KV8_INT8 && s.format != MOE_KV8_E4M3) return false;
  auto stride_ok = [](int v, long long least) { return v == 0 || (v % 8 == 0 && v >= least); };
  return stride_ok(s.q_stride, (long long)s.Hq * s.D) && stride_ok(s.kv_stride, (long long)s.Hkv * s.D);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool cache_ok(const moe_kv8_cache* c) {
  return c && c->k_codes && c->v_codes && c->k_scales && c->v_scales && aligned(c->k_codes, 16) &&
         aligned(c->v_codes, 16) && aligned(c->k_scales, 4) && aligned(c->v_scales, 4);
}

namespace {

template <int D, bool kE4m3>
void launch_write(const CacheArgs& p, int block, cudaStream_t s) {
  const dim3 grid((unsigned)(p.T / block + 2 * p.B), (unsigned)p.Hkv, 2u);
  if (block == 16) kv8_write_kernel<D, 16, kE4m3><<<grid, kThreads, 0, s>>>(p);
  else if (block == 32) kv8_write_kernel<D, 32, kE4m3><<<grid, kThreads, 0, s>>>(p);
  else kv8_write_kernel<D, 64, kE4m3><<<grid, kThreads, 0, s>>>(p);
}

template <int D, bool kE4m3>
void launch_read(const CacheArgs& p, int block, cudaStream_t s) {
  const dim3 grid((unsigned)((p.T + kReadTokens - 1) / kReadTokens), (unsigned)p.Hkv, 2u);
  if (block == 16) kv8_read_kernel<D, 16, kE4m3><<<grid, kThreads, 0, s>>>(p);
  else if (block == 32) kv8_read_kernel<D, 32, kE4m3><<<grid, kThreads, 0, s>>>(p);
  else kv8_read_kernel<D, 64, kE4m3><<<grid, kThreads, 0, s>>>(p);
}

moe_status cache_call(const moe_kv8_shape* shape, const moe_kv8_cache* cache, const int32_t* offsets,
                      const int32_t* starts, const void* k, const void* v, bool write, int32_t* status, void* stream) {
  if (!shape) return MOE_ERR_INVALID_ARG;
  const moe_kv8_shape s = *shape;
  if (!shape_ok(s)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!cache_ok(cache) || !aligned(offsets, 4) || !aligned(starts, 4) || !aligned(status, 4) || !aligned(k, 16) ||
      !aligned(v, 16))
    return MOE_ERR_INVALID_ARG;
  if (s.T == 0) return MOE_OK;
  if (!offsets || !starts || !k || !v) return MOE_ERR_INVALID_ARG;
  CacheArgs p{};
  p.codes[0] = cache->k_codes;
  p.codes[1] = cache->v_codes;
  p.scales[0] = cache->k_scales;
  p.scales[1] = cache->v_scales;
  if (write) {
    p.x[0] = static_cast<const uint16_t*>(k);
    p.x[1] = static_cast<const uint16_t*>(v);
  } else {
    p.out[0] = static_cast<uint16_t*>(const_cast<void*>(k));
    p.out[1] = static_cast<uint16_t*>(const_cast<void*>(v));
  }
  p.offsets = offsets;
  p.starts = starts;
  p.status = status;
  p.B = s.B;
  p.T = s.T;
  p.Hkv = s.Hkv;
  p.L_max = s.L_max;
  p.nblk = (s.L_max + s.block - 1) / s.block;
  p.stride = s.kv_stride ? s.kv_stride : s.Hkv * s.D;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = s.format == MOE_KV8_E4M3;
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (write) e4m3 ? launch_write<D, true>(p, s.block, st) : launch_write<D, false>(p, s.block, st);
    else e4m3 ? launch_read<D, true>(p, s.block, st) : launch_read<D, false>(p, s.block, st);
  };
  if (s.D == 64) go(std::integral_constant<int, 64>{});
  else if (s.D == 128) go(std::integral_constant<int, 128>{});
  else go(std::integral_constant<int, 256>{});
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, write ? "cache write launch" : "cache read launch");
}

}  // namespace
}  // namespace kv8
}  // namespace bgmoe

extern "C" {

moe_status moe_kv8_write(const moe_kv8_shape* shape, const void* k_new, const void* v_new, const int32_t* offsets,
                         const int32_t* starts, const moe_kv8_cache* cache, int32_t* status, void* stream) {
  return bgmoe::kv8::cache_call(shape, cache, offsets, starts, k_new, v_new, true, status, stream);
}

moe_status moe_kv8_read(const moe_kv8_shape* shape, const moe_kv8_cache* cache, const int32_t* offsets,
                        const int32_t* starts, void* k_out, void* v_out, int32_t* status, void* stream) {
  return bgmoe::kv8::cache_call(shape, cache, offsets, starts, k_out, v_out, false, status, stream);
}

}  // extern "C"
