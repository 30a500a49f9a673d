// Writing into and reading back from the 8-bit KV cache (include/kv8.h), sm_103a.
//
// Both move bytes and compute almost nothing: a value costs one multiply and
// one conversion, so they are bound by memory, and at a decode step's sizes
// by the latency of one dependent chain (tables, values, scale, codes).
// Measured (2 KV heads of 256, INT8, in a graph):
//   read of 32,768 positions  101 MB in 18.6 us, 5.4 TB/s, 80% of the measured
//                             copy rate; instructions take 53% of the issue slots
//   write of 4096 tokens, and 128 of them read back   8.7 us for 13 and 0.4 MB
//   write of a token of 64 sequences, and their open blocks read back   9.0 us
#include "kernels.h"
#include "kv8_attn.h"

#include <type_traits>

namespace bgmoe {
namespace kv8 {

constexpr int kThreads = 256;
// Its grid per SM, at most: as many blocks as a tile each would be 2048 for 32,768
// positions, each with the tables and the bisection in front of it: 30.7 us,
// against 19.6 with blocks that walk and ask for a tile ahead. (Of the larger
// tiles at 256 head dims, with 105 registers, two fit an SM at once: that grid
// runs in two waves.)
constexpr int kReadBlocks = 4;

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

// Launched with programmatic dependent launch: everything below may read what
// earlier kernels wrote or overwrite what they read, so it waits for them;
// then the next kernel's blocks may be set up (they wait in turn).
__device__ __forceinline__ void after_predecessors() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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
    const int lo = ld(p.offsets + b), hi = ld(p.offsets + b + 1), start = ld(p.starts + b);
    if (offsets_bad(lo, hi, b, p.B, p.T) || range_bad(start, hi - lo, p.L_max)) bad = true;
    else hit(b, lo, hi, start);
  }
  return __syncthreads_or(bad) != 0;
}

// A unit of work is one touched cache block of one KV head, K or V. Sequence b's
// touched blocks are numbered floor(offsets[b] / kBlock) + 2 b + 0, 1, ...: n
// tokens touch at most floor(n / kBlock) + 2 blocks, which is what the next
// sequence's first number leaves room for, so no prefix sum is needed and there
// are floor(T / kBlock) + 2 B numbers (some of them touch nothing).
//
// A unit has 64 values per thread, kPer 16-byte pieces, which stay in registers
// between the maximum and the codes, so they are read once, with all loads in
// flight together: a warp for a block of 16 x 64 values, the whole thread block
// of 256 for one of 64 x 256. The rare values that are not finite are read
// again instead, in loops of their own: 80 registers for 128, so that three
// thread blocks fit an SM. 5617 tokens of 5 sequences, 8 heads of 128, written
// and read back: 20.9 -> 16.0 us.
template <int D, int kBlock>
struct WriteCfg {
  static constexpr int kUnitThreads = kBlock * D / 64 < 32 ? 32 : kBlock * D / 64;
  static constexpr int kUnits = kThreads / kUnitThreads;              // units of a thread block
  static constexpr int kPer = kBlock * D / 8 / kUnitThreads;          // pieces of a thread
};

template <int D, int kBlock, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 3) kv8_write_kernel(const CacheArgs p) {
  using W = WriteCfg<D, kBlock>;
  constexpr int kPer = W::kPer, kTU = W::kUnitThreads;
  __shared__ int s_b[W::kUnits], s_lo[W::kUnits], s_n[W::kUnits], s_start[W::kUnits];
  __shared__ uint32_t s_max[2][kThreads / 32];
  after_predecessors();
  // units in the order (number, head, K or V)
  const int per = 2 * p.Hkv, first = blockIdx.x * W::kUnits, local = threadIdx.x / kTU, tu = threadIdx.x % kTU;
  const int item = first + local, unit = item / per, g = (item - unit * per) >> 1, kv = item & 1;
  if (threadIdx.x < W::kUnits) s_b[threadIdx.x] = -1;
  __syncthreads();
  const bool bad = tables_bad(p, [&](int b, int lo, int hi, int start) {
    const int u0 = lo / kBlock + 2 * b, u1 = hi / kBlock + 2 * (b + 1);
    if (u1 <= first / per || u0 > (first + W::kUnits - 1) / per) return;
    for (int k = 0; k < W::kUnits; ++k) {
      const int u = (first + k) / per;
      if (u >= u0 && u < u1) {
        s_b[k] = b;
        s_lo[k] = lo;
        s_n[k] = hi - lo;
        s_start[k] = start;
      }
    }
  });
  if (bad) {
    if (threadIdx.x == 0) flag(p.status, (int32_t)MOE_ERR_INVALID_ARG);
    return;
  }
  const int b = s_b[local];
  const int n = b < 0 ? 0 : s_n[local], start = b < 0 ? 0 : s_start[local], lo = b < 0 ? 0 : s_lo[local];
  const int blk = start / kBlock + (unit - (lo / kBlock + 2 * b));
  const int base = blk * kBlock;                       // the cache block's first position
  const int p0 = max(start, base), p1 = min(start + n, base + kBlock);  // its new positions
  // The threads of a unit share everything up to here, so a unit without new
  // positions takes no part in the others' barriers.
  if (b < 0 || n == 0 || p0 >= p1) return;
  const size_t pair = (size_t)b * p.Hkv + g;
  uint8_t* codes = (kv ? p.codes[1] : p.codes[0]) + (pair * p.L_max + base) * D;
  float* scale = (kv ? p.scales[1] : p.scales[0]) + pair * p.nblk + blk;
  const int r0 = p0 - base, r1 = p1 - base;            // rows of the block
  const uint16_t* x = (kv ? p.x[1] : p.x[0]) + (size_t)(lo + (p0 - start)) * p.stride + (size_t)g * D;  // of row r0

  uint4 v[kPer];
  uint32_t mx = 0;  // largest magnitude bits, two bf16 side by side
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int piece = tu + i * kTU;                    // piece of the new rows, from row r0
    const int row = piece / (D / 8), c = piece % (D / 8);
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < r1 - r0) v[i] = ld_once_v4(x + (size_t)row * p.stride + c * 8);
  }
  const float s_old = p0 > base ? *scale : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, w[j] & 0x7FFF7FFFu);
  }
  // Over both halves and all threads of the unit; a barrier of the unit's own
  // (its threads have all read s_old when it is passed).
  auto unit_max = [&](uint32_t m2, int turn) -> uint32_t {
    uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
    if (kTU > 32) {
      if ((threadIdx.x & 31) == 0) s_max[turn][threadIdx.x >> 5] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(local + 1), "n"(kTU) : "memory");
#pragma unroll
      for (int w = 0; w < kTU / 32; ++w) m = max(m, s_max[turn][local * (kTU / 32) + w]);
    }
    return m;
  };
  uint32_t m = unit_max(mx, 0);
  // Rare values: an infinity or a NaN (the maximum again over finite values, and
  // they are replaced); in E4M3, from 1.9375 * 2^127 on, those next to code 256 of
  // the scale 2^120, whose value is 2^128: they take 240, which is nearer than half
  // a step of theirs (2^-4).
  constexpr uint32_t kTop = kE4m3 ? 0x7F77u : 0x7F7Fu;
  const bool odd = m > kTop;
  auto reload = [&](int piece) { return ld_once_v4(x + (size_t)(piece / (D / 8)) * p.stride + piece % (D / 8) * 8); };
  const int pieces = (r1 - r0) * (D / 8);
  if (odd) {
    if (tu == 0 && m >= 0x7F80u) flag(p.status, (int32_t)MOE_ERR_RANGE);
    mx = 0;
#pragma unroll 1
    for (int piece = tu; piece < pieces; piece += kTU) {
      const uint4 y = reload(piece);
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo2 = w[j] & 0x7FFFu, hi2 = (w[j] >> 16) & 0x7FFFu;
        mx = __vmaxu2(mx, (lo2 < 0x7F80u ? lo2 : 0u) | (hi2 < 0x7F80u ? hi2 : 0u) << 16);
      }
    }
    m = unit_max(mx, 1);
  }
  const float s_new = fmaxf(s_old, scale_of<kE4m3>(__uint_as_float(m << 16)));
  const float inv = inverse_scale(s_new);
  if (p0 > base && s_new > s_old) {  // the block's earlier codes, to the larger scale
    for (int piece = tu; piece < r0 * (D / 4); piece += kTU) {
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
  if (kTU == 32) __syncwarp();  // s_old has been read by all
  if (tu == 0 && (p0 == base || s_new != s_old)) *scale = s_new;
  // 8 new values to codes (the new rows' codes follow one another)
  auto put = [&](int piece, const uint32_t (&w)[4]) {
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float f0 = __uint_as_float(w[2 * j] << 16), f1 = __uint_as_float(w[2 * j] & 0xFFFF0000u);
      const float f2 = __uint_as_float(w[2 * j + 1] << 16), f3 = __uint_as_float(w[2 * j + 1] & 0xFFFF0000u);
      o[j] = encode4<kE4m3>(f0 * inv, f1 * inv, f2 * inv, f3 * inv);
    }
    *reinterpret_cast<uint2*>(codes + (size_t)r0 * D + (size_t)piece * 8) = make_uint2(o[0], o[1]);
  };
  if (odd) {
    auto finite = [&](uint32_t h) -> uint32_t {  // one bf16
      const uint32_t a = h & 0x7FFFu;
      return a > 0x7F80u ? 0u : (h & 0x8000u) | min(a == 0x7F80u ? m : a, kTop);
    };
#pragma unroll 1
    for (int piece = tu; piece < pieces; piece += kTU) {
      const uint4 y = reload(piece);
      uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = finite(w[j] & 0xFFFFu) | finite(w[j] >> 16) << 16;
      put(piece, w);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    if (tu + i * kTU < pieces) put(tu + i * kTU, w);
  }
}

// Thread blocks walk over tiles of kReadTokens packed tokens of one KV head, K or V. The
// tables are checked once; a tile's tokens find their sequence and position
// (by bisection of the offsets), then each thread turns 8-byte pieces of codes
// into 16 bytes of bf16, so a warp's stores fill whole sectors. The next tile's
// codes are asked for before this one's are converted.
template <int D, int kBlock, bool kE4m3, int kReadTokens>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const CacheArgs p) {
  constexpr int kRow = D / 8;                           // pieces per token
  constexpr int kPer = kReadTokens * kRow / kThreads;   // pieces per thread
  __shared__ long long s_code[2][kReadTokens];          // first code of each token (head g), in bytes
  __shared__ long long s_scale[2][kReadTokens];         // its scale
  after_predecessors();
  if (tables_bad(p, [](int, int, int, int) {})) {
    if (threadIdx.x == 0) flag(p.status, (int32_t)MOE_ERR_INVALID_ARG);
    return;
  }
  const int per = 2 * p.Hkv, tiles = (p.T + kReadTokens - 1) / kReadTokens * per;
  auto find = [&](int tile, int buf) {                  // by the first kReadTokens threads
    const int t = tile / per * kReadTokens + threadIdx.x, g = (tile % per) >> 1;
    if (threadIdx.x >= kReadTokens || t >= p.T) return;
    int b = 0, z = p.B;                                 // the last sequence that starts at or before t
    while (z - b > 1) {
      const int mid = (b + z) >> 1;
      if (ld(p.offsets + mid) <= t) b = mid;
      else z = mid;
    }
    const int pos = ld(p.starts + b) + t - ld(p.offsets + b);
    const long long pair = (long long)b * p.Hkv + g;
    s_code[buf][threadIdx.x] = (pair * p.L_max + pos) * D;
    s_scale[buf][threadIdx.x] = pair * p.nblk + pos / kBlock;
  };
  uint2 w[kPer];
  float s[kPer];
  auto load = [&](int tile, int buf) {
    const int nt = min(kReadTokens, p.T - tile / per * kReadTokens);
    const uint8_t* codes = tile & 1 ? p.codes[1] : p.codes[0];
    const float* scales = tile & 1 ? p.scales[1] : p.scales[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int piece = threadIdx.x + i * kThreads, t = piece / kRow, c = piece % kRow;
      w[i] = make_uint2(0, 0);
      s[i] = 0.f;
      if (t < nt) {
        w[i] = __ldcs(reinterpret_cast<const uint2*>(codes + s_code[buf][t] + c * 8));
        s[i] = ld(scales + s_scale[buf][t]);
      }
    }
  };
  int tile = blockIdx.x, buf = 0;
  if (tile >= tiles) return;
  find(tile, 0);
  __syncthreads();
  load(tile, 0);
  for (; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int next = tile + gridDim.x, t0 = tile / per * kReadTokens, g = (tile % per) >> 1;
    uint16_t* out = tile & 1 ? p.out[1] : p.out[0];
    if (next < tiles) find(next, buf ^ 1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int piece = threadIdx.x + i * kThreads, t = piece / kRow, c = piece % kRow;
      if (t0 + t >= p.T) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[4];
        decode4<kE4m3>(j ? w[i].y : w[i].x, f);
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0] * s[i], f[1] * s[i]);
        const __nv_bfloat162 z = __floats2bfloat162_rn(f[2] * s[i], f[3] * s[i]);
        o[2 * j] = *reinterpret_cast<const uint32_t*>(&a);
        o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&z);
      }
      __stcs(reinterpret_cast<uint4*>(out + ((size_t)(t0 + t) * p.Hkv + g) * D + c * 8),
             make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (next < tiles) load(next, buf ^ 1);
  }
}

// ================================================================= host ===

bool shape_ok(const moe_kv8_shape& s) {
  if (s.B < 1 || s.B > 4096 || s.T < 0 || s.T > (1 << 24)) return false;
  if (s.Hkv < 1 || s.Hkv > 4096 || s.Hq < 1 || s.Hq % s.Hkv != 0 || (long long)s.T * s.Hkv > (1 << 30)) return false;
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

template <typename Kernel>
cudaError_t launch(Kernel kernel, long long grid, const CacheArgs& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int kBlock, bool kE4m3>
cudaError_t launch_one(const CacheArgs& p, bool write, int sms, cudaStream_t s) {
  if (write) {
    const long long items = ((long long)p.T / kBlock + 2 * p.B) * 2 * p.Hkv;
    constexpr int kUnits = WriteCfg<D, kBlock>::kUnits;
    return launch(kv8_write_kernel<D, kBlock, kE4m3>, (items + kUnits - 1) / kUnits, p, s);
  }
  // Tiles of 64 tokens, or larger ones where those fill the grid as well (64
  // and larger, in us): 1000 tokens of 2 sequences, one head of 64, 2.2 and 3.0;
  // 131,072 tokens of such a head 12.3 and 9.5; 12,000 of 8 heads of 128 17.0
  // and 14.7; 32,768 of 2 heads of 256 19.3 and 18.7.
  constexpr int kSmall = 64, kLarge = D == 64 ? 256 : 128;
  auto tiles = [&](int tokens) { return (long long)((p.T + tokens - 1) / tokens) * 2 * p.Hkv; };
  const long long most = (long long)sms * kReadBlocks;
  if (tiles(kLarge) >= most) return launch(kv8_read_kernel<D, kBlock, kE4m3, kLarge>, most, p, s);
  return launch(kv8_read_kernel<D, kBlock, kE4m3, kSmall>, tiles(kSmall) < most ? tiles(kSmall) : most, p, s);
}

template <int D, bool kE4m3>
cudaError_t launch_block(const CacheArgs& p, bool write, int block, int sms, cudaStream_t s) {
  return block == 16   ? launch_one<D, 16, kE4m3>(p, write, sms, s)
         : block == 32 ? launch_one<D, 32, kE4m3>(p, write, sms, s)
                       : launch_one<D, 64, kE4m3>(p, write, sms, s);
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
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice, "device query");
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return e4m3 ? launch_block<D, true>(p, write, s.block, sms, st)
                : launch_block<D, false>(p, write, s.block, sms, st);
  };
  const cudaError_t e = s.D == 64    ? go(std::integral_constant<int, 64>{})
                        : s.D == 128 ? go(std::integral_constant<int, 128>{})
                                     : go(std::integral_constant<int, 256>{});
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
