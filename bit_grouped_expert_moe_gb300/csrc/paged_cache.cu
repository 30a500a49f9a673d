// Writing the paged cache (include/paged.h): appending new tokens, and moving
// the accepted drafts of a tree behind the context.
//
// Append is the pass of rope.cuh over queries, keys and values; keys and values
// go to the token's row of a page. The chain offsets -> start -> page is what a decode step
// waits for, so the token's sequence is guessed first (token t is sequence t's
// where every sequence has one) and searched for only where the guess is wrong.
#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "paged_path.h"
#include "rope.cuh"

namespace bgmoe {
namespace paged {

bool shape_ok(const moe_paged_shape& s) {
  if (s.B < 1 || s.B > 4096 || s.T < 0 || s.T > (1 << 24)) return false;
  if (s.Hkv < 1 || s.Hkv > 4096 || s.Hq < 1 || s.Hq % s.Hkv != 0 || (long long)s.T * s.Hkv > (1 << 30)) return false;
  if (s.Hq / s.Hkv > 64 || (long long)s.B * s.Hkv > 65536) return false;
  if (s.D != 64 && s.D != 128 && s.D != 256) return false;
  if (s.page != 16 && s.page != 32 && s.page != 64 && s.page != 128 && s.page != 256) return false;
  if (s.n_pages < 1 || (long long)s.n_pages * s.Hkv > 0x7FFFFFFFll) return false;
  if (s.max_pages < 1 || (long long)s.max_pages * s.page > (1 << 26)) return false;
  if (s.tree_words < 0 || s.tree_words > 8) return false;
  const auto stride_ok = [](int v, long long least) { return v == 0 || (v % 8 == 0 && v >= least); };
  return stride_ok(s.q_stride, (long long)s.Hq * s.D) && stride_ok(s.kv_stride, (long long)s.Hkv * s.D);
}

bool cache_ok(const moe_paged_cache* c) {
  return c && c->k_pages && c->v_pages && c->tables && aligned(c->k_pages, 16) && aligned(c->v_pages, 16) &&
         aligned(c->tables, 4);
}

namespace {

constexpr int kAhead = 4, kBlocks = 6;  // as in rope.cu

struct Append {
  const uint16_t* q;
  const uint16_t* kv[2];
  uint16_t* q_out;
  uint16_t* pages[2];
  const int32_t* offsets;
  const int32_t* starts;
  const int32_t* positions;
  const int32_t* tables;
  int32_t* status;
  long long qs, kvs;  // elements from token to token
  int B, Hq, Hkv, D, shift, n_pages, max_pages;  // Hq = 0 without queries
  struct Token {
    long long row;  // of KV head 0 in the pools
  };
  // The token's sequence and its position there; false where the tables break
  // the rules for it.
  __device__ bool token(int t, Token* k, int* position) const {
    int b = min(t, B - 1);
    int lo = ld(offsets + b), hi = ld(offsets + b + 1), start = ld(starts + b);
    if (t < lo || t >= hi) {
      // the last sequence that starts at or before t
      int a = 0, z = B;
      while (z - a > 1) {
        const int m = (a + z) >> 1;
        if (ld(offsets + m) <= t) a = m;
        else z = m;
      }
      b = a;
      lo = ld(offsets + b);
      hi = ld(offsets + b + 1);
      start = ld(starts + b);
    }
    const long long pos = (long long)start + (t - (long long)lo);
    if (lo < 0 || t < lo || t >= hi || start < 0 || pos >= ((long long)max_pages << shift)) return false;
    const int page = ld(tables + (long long)b * max_pages + (pos >> shift));
    if (page < 0 || page >= n_pages) return false;
    k->row = ((long long)page * Hkv << shift) + (pos & ((1 << shift) - 1));
    *position = positions != nullptr ? ld(positions + t) : (int)pos;
    return true;
  }
  __device__ int kind(int h) const { return h < Hq ? 0 : h < Hq + Hkv ? 1 : 2; }
  __device__ const uint16_t* from(int t, int h) const {
    const int j = h - Hq;
    return j < 0      ? q + t * qs + (long long)h * D
           : j < Hkv ? kv[0] + t * kvs + (long long)j * D
                     : kv[1] + t * kvs + (long long)(j - Hkv) * D;
  }
  __device__ uint16_t* to(const Token& k, int t, int h) const {
    const int j = h - Hq;
    return j < 0      ? q_out + ((long long)t * Hq + h) * D
           : j < Hkv ? pages[0] + (k.row + ((long long)j << shift)) * D
                     : pages[1] + (k.row + ((long long)(j - Hkv) << shift)) * D;
  }
  __device__ void refuse() const {
    if (status != nullptr) atomicCAS(status, 0, (int32_t)MOE_ERR_INVALID_ARG);
  }
};

template <int kLanes>
__global__ void __launch_bounds__(rope::kThreads, kBlocks)
    paged_append_kernel(const Append io, const rope::Spec spec, const rope::Split split) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  rope::turn<kLanes, kAhead>(io, spec, split);
}

// ------------------------------------------------------------------ keep ---

constexpr int kMaxPath = 512;
constexpr int kKeepThreads = 128;
// Rows in flight per thread. us for 200 sequences of 20 to 40 rows of 8 heads of 128,
// and 1000 of 9: 4 11.1 and 8.8; 8 10.8 and 9.2; 10 8.4 and 8.3; 12 8.4 and 8.5; 14 7.9
// and 8.6; 16 10.0 and 9.9; 20 8.1 and 10.0.
constexpr int kRowsAhead = 14;

struct KeepParams {
  uint16_t* pages[2];
  const int32_t* tables;
  const int32_t* starts;
  const int32_t* kept;
  const int32_t* path;
  int32_t* lens_out;
  int32_t* status;
  int path_stride, Hkv, D, shift, n_pages, max_pages;
};

// Block (b, y): sequence b, the y-th 128 of its 2 Hkv D / 8 columns of 16
// bytes, a thread each. Row k comes from row path[k] >= k, and the rows are
// read in order, so a row is never written before all that read it have: a
// thread may read as far ahead as it likes, and columns do not meet.
// Bound: the chain kept and start -> path -> pages -> rows (64 sequences of up
// to 8 kept rows 2.5 us in a graph); the rows themselves are read and written once.
__global__ void __launch_bounds__(kKeepThreads) paged_keep_kernel(const KeepParams p) {
  __shared__ long long s_row[2][kMaxPath];  // from, to: rows of the pools at KV head 0, in rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x, t = threadIdx.x;
  const int start = ld(p.starts + b), kept = ld(p.kept + b);
  bool bad = start < 0 || kept < 0 || kept > p.path_stride;
  const long long limit = (long long)p.max_pages << p.shift;
  bad = bad || start > limit;
  if (!bad) {
    for (int k = t; k < kept; k += kKeepThreads) {
      const int32_t* path = p.path + (long long)b * p.path_stride + k;
      const int from = ld(path), before = k > 0 ? ld(path - 1) : -1;
      if (!path_entry_ok(from, before, k, start, limit)) {
        bad = true;
        continue;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int pos = start + (e ? k : from);
        const int page = ld(p.tables + (long long)b * p.max_pages + (pos >> p.shift));
        if (page < 0 || page >= p.n_pages) bad = true;
        s_row[e][k] = ((long long)page * p.Hkv << p.shift) + (pos & ((1 << p.shift) - 1));
      }
    }
  }
  if (__syncthreads_or(bad)) {
    if (t == 0 && blockIdx.y == 0 && p.status != nullptr) atomicCAS(p.status, 0, (int32_t)MOE_ERR_INVALID_ARG);
    return;
  }
  if (t == 0 && blockIdx.y == 0 && p.lens_out != nullptr) p.lens_out[b] = start + kept;
  const int half = p.Hkv * (p.D / 8), c = blockIdx.y * kKeepThreads + t;
  if (c >= 2 * half) return;
  const int v = c >= half, in = v ? c - half : c, h = in / (p.D / 8), d = (in % (p.D / 8)) * 8;
  uint16_t* base = (v ? p.pages[1] : p.pages[0]) + ((long long)h << p.shift) * p.D + d;
  for (int k0 = 0; k0 < kept; k0 += kRowsAhead) {
    uint4 x[kRowsAhead];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i)
      if (k0 + i < kept && s_row[0][k0 + i] != s_row[1][k0 + i])
        x[i] = ld_once_v4(base + s_row[0][k0 + i] * p.D);
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i)
      if (k0 + i < kept && s_row[0][k0 + i] != s_row[1][k0 + i])
        *reinterpret_cast<uint4*>(base + s_row[1][k0 + i] * p.D) = x[i];
  }
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace
}  // namespace paged
}  // namespace bgmoe

extern "C" {

moe_status moe_paged_append(const moe_paged_shape* shape, const moe_rope_spec* spec, const void* q, const void* k_new,
                            const void* v_new, const int32_t* offsets, const int32_t* starts, const int32_t* positions,
                            const moe_paged_cache* cache, void* q_out, int32_t* status, void* stream) {
  using namespace bgmoe;
  using namespace bgmoe::paged;
  if (!shape) return MOE_ERR_INVALID_ARG;
  const moe_paged_shape s = *shape;
  if (!shape_ok(s) || (spec && !rope::spec_ok(*spec, s.D))) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!cache_ok(cache) || !aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(offsets, 4) || !aligned(starts, 4) || !aligned(positions, 4) || !aligned(status, 4) ||
      (spec && !rope::spec_pointers_ok(*spec)) || (q == nullptr) != (q_out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (s.T == 0) return MOE_OK;
  if (!k_new || !v_new || !offsets || !starts) return MOE_ERR_INVALID_ARG;
  const int Hq = q ? s.Hq : 0;
  const Append io{static_cast<const uint16_t*>(q),
                  {static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new)},
                  static_cast<uint16_t*>(q_out),
                  {static_cast<uint16_t*>(cache->k_pages), static_cast<uint16_t*>(cache->v_pages)},
                  offsets, starts, positions, cache->tables, status,
                  s.q_stride ? s.q_stride : (long long)s.Hq * s.D, s.kv_stride ? s.kv_stride : (long long)s.Hkv * s.D,
                  s.B, Hq, s.Hkv, s.D, page_shift(s.page), s.n_pages, s.max_pages};
  long long blocks = 0;
  const rope::Split sl = rope::split(s.T, Hq + 2 * s.Hkv, s.D, spec ? spec->rot : 0, kAhead, &blocks);
  const int lanes = rope::head_lanes(s.D);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      config(dim3((unsigned)blocks), rope::kThreads, static_cast<cudaStream_t>(stream), &attr);
  const auto go = [&](auto n) {
    return cudaLaunchKernelEx(&cfg, paged_append_kernel<decltype(n)::value>, io, rope::device_spec(spec), sl);
  };
  const cudaError_t e = lanes == 4   ? go(std::integral_constant<int, 4>{})
                        : lanes == 8 ? go(std::integral_constant<int, 8>{})
                                     : go(std::integral_constant<int, 16>{});
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "append launch");
}

moe_status moe_paged_keep(const moe_paged_shape* shape, const moe_paged_cache* cache, const int32_t* starts,
                          const int32_t* kept, const int32_t* path, int32_t path_stride, int32_t* lens_out,
                          int32_t* status, void* stream) {
  using namespace bgmoe;
  using namespace bgmoe::paged;
  if (!shape) return MOE_ERR_INVALID_ARG;
  const moe_paged_shape s = *shape;
  if (!shape_ok(s) || path_stride < 0 || path_stride > kMaxPath) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!cache_ok(cache) || !aligned(starts, 4) || !aligned(kept, 4) || !aligned(path, 4) || !aligned(lens_out, 4) ||
      !aligned(status, 4) || !starts || !kept || (path_stride > 0 && !path))
    return MOE_ERR_INVALID_ARG;
  const KeepParams p{{static_cast<uint16_t*>(cache->k_pages), static_cast<uint16_t*>(cache->v_pages)},
                     cache->tables, starts, kept, path, lens_out, status, path_stride, s.Hkv, s.D,
                     page_shift(s.page), s.n_pages, s.max_pages};
  const int columns = 2 * s.Hkv * (s.D / 8);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      config(dim3((unsigned)s.B, (unsigned)((columns + kKeepThreads - 1) / kKeepThreads)), kKeepThreads,
             static_cast<cudaStream_t>(stream), &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_keep_kernel, p);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "keep launch");
}

}  // extern "C"
