// Attention over the 8-bit KV cache for many query tokens per sequence
// (prompts, chunks of prompts), on the 5th-generation tensor cores, sm_103a.
//
// A row is one (query token, query head of a KV head); a row tile is 128
// consecutive rows of one (sequence, KV head), so the query heads that share
// keys share a tile whatever Hq / Hkv is. The positions that a tile's last
// row sees are cut into units of 128, and all units of the call, laid end to
// end in the order (sequence, KV head, row tile, position), are dealt out in
// equal contiguous runs, one per block of a one-block-per-SM grid: a triangle
// of causal tiles and a few tiles over a long context both fill every SM. A
// tile that lies in one run is finished by its block; one that a run's border
// cuts leaves partial states (m, L, O) in the workspace, at most two per
// block, which kv8_tiles_merge_kernel joins in a fixed order.
//
// Per unit and tile, 4 * 128 * 128 * D flops:
//   S = Q K^T  128 x 128 x D, both operands in shared memory, S in TMEM;
//   P = 2^(x - m + 7) in fp16, written over S in TMEM;
//   O += P V   128 x D x 128, A = P from TMEM, B = V from shared memory as it
//              lies in the cache, position by position (an MN-major operand).
// S is double buffered, so the product S of the next unit runs while the
// softmax of this one is computed (TMEM: D columns of O, 2 x 128 of S).
//
// Warp roles (512 threads):
//   warp 0       TMEM allocation and the single MMA-issuing thread
//   warps 4-7    softmax: thread = row (TMEM lane); at a tile's end the output
//   warps 8-15   codes -> fp16 operands: 16-byte global loads two ring stages
//                ahead in registers, converted and stored with the 128-byte
//                swizzle; they also bring Q in (bf16 -> fp16, row by row)
// The ring's stages are 128 positions x 128 head dims of K or 64 x 256 of V
// (32 KB of fp16) and come in the order the MMAs use them: K of unit u + 1,
// then V of unit u.
//
// Codes and scales as in kv8_split.cu: int8 K enters as u 2^-24 (u = code +
// 128, an fp16 subnormal, one byte permute per pair) and the row's constant
// 128 sum(q) comes off in the fused multiply-add that applies the scales; V is
// exact; with x = score + log2 s_v the weights carry V's scale and
// L = sum w / s_v. The running maximum m of a row is raised only when a score
// passes it by more than 8 (on the base-2 scale), so that O in TMEM is
// rarely rescaled: w <= 2^15.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "kv8_attn.h"
#include "tc_ptx.cuh"

namespace bgmoe {
namespace kv8 {
namespace tiles {

using namespace tc;

constexpr int kRows = 128;          // rows of a tile (MMA M)
constexpr int kKeys = 128;          // positions of a unit
constexpr int kThreads = 512;
constexpr int kConvWarps = 8;
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kMaxCtas = 256;       // workspace bound on the grid
constexpr long long kTimeoutNs = 1000000000ll;
constexpr float kMinusBig = -1e30f;
constexpr float kWeightBits = 7.f;  // weights are 2^7 at the row's m ...
constexpr float kSlack = 8.f;       // ... which scores may pass by this much
constexpr int kTmemCols = 512;
constexpr uint32_t kColS = 256;     // S buffers at columns 256 and 384, O from 0

template <int D>
struct Cfg {
  static constexpr int kKParts = D > 128 ? D / 128 : 1;  // ring stages of a unit's K ...
  static constexpr int kKDims = D / kKParts;             // ... by head dims
  static constexpr int kVParts = D > 128 ? D / 128 : 1;  // ... and of its V
  static constexpr int kVKeys = kKeys / kVParts;         // ... by positions
  static constexpr int kStageBytes = kKeys * kKDims * 2; // = kVKeys * D * 2
  static constexpr int kStages = D == 64 ? 8 : 4;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kLoads = kStageBytes / 2 / 16 / kConvThreads;  // 16-byte loads per thread and stage
  static constexpr int kCtlOffset = kQBytes + kStages * kStageBytes;
  static constexpr int kBytes = kCtlOffset + 4096 + 1024;  // + alignment slack
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct RowConst {  // of a tile's rows, written with its Q
  float scale[kRows];   // scale * log2(e) * 2^e, e the row's power of two
  float shift[kRows];   // -128 sum(q) 2^-24 (int8)
  int see[kRows];       // visible positions (0 for rows past the last)
};

template <int kStages>
struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t rc_full[2], rc_empty[2];  // row constants of every second tile
  uint64_t s_full[2], p_full[2];
  // One arrival per unit, on alternate barriers. A waiter's parity is safe if
  // it cannot be two phases off: the softmax of unit u has seen S of unit u,
  // whose commit covers the products of u - 2, and those of u + 1 and u + 2
  // wait for its weights.
  uint64_t pv_done[2];
  uint64_t o_empty;       // O of a finished tile has been read
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
  RowConst rc[2];
};

struct RunInfo {  // where a block's run starts, for the merge kernel
  long long units;  // units of the call (0: nothing to do or bad tables)
  long long lo;     // the run's first unit
  int b, g, rt, i, nb;
  int live;         // the run is not empty
};

struct Params {
  const uint16_t* q;
  const uint8_t* codes[2];  // K, V
  const float* ks;
  const float* vs;
  const int32_t* offsets;
  const int32_t* lens;
  uint16_t* o;
  float* part;       // [2 C] slots of [D][128] O, then [128] m, [128] L
  RunInfo* info;     // [C]
  int32_t* flags;    // [C]
  float scale_log2;
  int B, T, Hq, Hkv, L_max, nblk, shift, q_stride;
  long long timeout_ns;
};

constexpr size_t slot_floats(int D) { return (size_t)kRows * (D + 2); }

// Place in the run: unit i of the nb units of row tile rt of KV head g of
// sequence b.
struct Cursor {
  int b, g, rt, i, nb, n, len, lo;
  __device__ void sequence(const Params& p) {
    lo = __ldg(p.offsets + b);
    n = __ldg(p.offsets + b + 1) - lo;
    len = __ldg(p.lens + b);
  }
  __device__ bool first() const { return i == 0; }
  __device__ bool last() const { return i == nb - 1; }
  __device__ void advance(const Params& p, int r) {
    if (++i < nb) return;
    i = 0;
    do {
      if (++rt >= seq_tiles(n, r, kRows)) {
        rt = 0;
        if (++g >= p.Hkv) {
          g = 0;
          do {
            if (++b >= p.B) return;
            sequence(p);
          } while (n == 0);
        }
      }
      nb = tile_units(n, len, r, kRows, kKeys, rt);
    } while (nb == 0);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an MN-major operand in the 128-byte swizzle: 64 values along
// N per 128-byte row, one row per position, 8-row atoms of 1024 bytes along K
// (stride offset), the next 64 values of N `block` bytes on (leading offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((block >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four codes as four fp16 values in order. int8: K as u 2^-24, V as the code.
template <bool kE4m3, bool kV>
__device__ __forceinline__ void convert4(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (kE4m3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p01) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p23) : "h"((uint16_t)(w >> 16)));
  } else if (kV) {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    p01 = *reinterpret_cast<const uint32_t*>(&x);
    p23 = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    p01 = __byte_perm(w, 0u, 0x4140);
    p23 = __byte_perm(w, 0u, 0x4342);
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) kv8_tiles_kernel(const Params p) {
  using F = Cfg<D>;
  constexpr int kStages = F::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // 64-dim slabs of 128 rows x 128 bytes
  uint8_t* sR = smem + F::kQBytes;     // ring
  Ctl<kStages>* ctl = reinterpret_cast<Ctl<kStages>*>(smem + F::kCtlOffset);
  static_assert(sizeof(Ctl<kStages>) <= 4096, "control block");
  __shared__ long long s_lo, s_hi;
  __shared__ Cursor s_cur;
  __shared__ int s_bad;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = gridDim.x, c = blockIdx.x;
  const int r = p.Hq / p.Hkv;

  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], kConvWarps);
      mbar_init(&ctl->empty[s], 1);
    }
    mbar_init(&ctl->q_full, kConvWarps);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->rc_full[i], kConvWarps);
      mbar_init(&ctl->rc_empty[i], 4);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->pv_done[i], 1);
    }
    mbar_init(&ctl->o_empty, 4);
    mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  // Launched with programmatic dependent launch: wait for the kernels before
  // this one, then let this call's merge launch (it waits in turn).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 1) {
    // Check the tables, count the units and find where this block's run starts.
    long long total = 0;
    bool bad = false;
    for (int base = 0; base < p.B; base += 32) {
      const int b = base + lane;
      long long v = 0;
      if (b < p.B) {
        const int lo = __ldg(p.offsets + b), hi = __ldg(p.offsets + b + 1), len = __ldg(p.lens + b);
        if (offsets_bad(lo, hi, b, p.B, p.T) || len < 0 || len > p.L_max) bad = true;
        else v = units_before(hi - lo, len, r, kRows, kKeys, seq_tiles(hi - lo, r, kRows));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      total += v;
    }
    bad = __any_sync(0xffffffffu, bad);
    total *= p.Hkv;
    const long long lo = (long long)c * total / C, hi = (long long)(c + 1) * total / C;
    Cursor k{};
    if (!bad && lo < hi) {
      long long acc = 0, off = 0, per = 0;
      for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        long long v = 0;
        if (b < p.B) {
          const int n = __ldg(p.offsets + b + 1) - __ldg(p.offsets + b);
          v = units_before(n, __ldg(p.lens + b), r, kRows, kKeys, seq_tiles(n, r, kRows)) * p.Hkv;
        }
        long long incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, acc + incl > lo);
        if (hit) {
          const int L = __ffs(hit) - 1;
          k.b = base + L;
          off = lo - (acc + __shfl_sync(0xffffffffu, incl - v, L));
          per = __shfl_sync(0xffffffffu, v, L) / p.Hkv;
          break;
        }
        acc += __shfl_sync(0xffffffffu, incl, 31);
      }
      k.sequence(p);
      k.g = (int)(off / per);
      off -= k.g * per;
      // the last tile whose first unit is at or before off, 32 candidates a round
      int a = 0, z = seq_tiles(k.n, r, kRows);
      while (z - a > 1) {
        const int step = (z - a + 31) / 32, cand = a + lane * step;
        const bool in = cand < z && units_before(k.n, k.len, r, kRows, kKeys, cand) <= off;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));
        a += last * step;
        z = min(z, a + step);
      }
      // tiles without units share their successor's first unit: the search
      // ends on the last of them, which has some
      k.rt = a;
      k.i = (int)(off - units_before(k.n, k.len, r, kRows, kKeys, a));
      k.nb = tile_units(k.n, k.len, r, kRows, kKeys, a);
    }
    if (lane == 0) {
      s_lo = lo;
      s_hi = hi;
      s_bad = bad;
      s_cur = k;
      p.info[c] = RunInfo{bad ? 0 : total, lo, k.b, k.g, k.rt, k.i, k.nb, !bad && lo < hi};
    }
  }
  __syncthreads();
  if (s_bad) {
    if (threadIdx.x == 0) p.flags[c] = (int32_t)MOE_ERR_INVALID_ARG;
    return;
  }
  // Queries that see nothing (more queries than positions): o = 0.
  for (int b = c; b < p.B; b += C) {
    const int lo = __ldg(p.offsets + b), hi = __ldg(p.offsets + b + 1), len = __ldg(p.lens + b);
    const size_t pieces = (size_t)max(0, hi - lo - len) * p.Hq * (D / 8);
    uint4* z = reinterpret_cast<uint4*>(p.o + (size_t)lo * p.Hq * D);
    for (size_t i = threadIdx.x; i < pieces; i += kThreads) z[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (s_lo >= s_hi) {
    if (threadIdx.x == 0) p.flags[c] = 0;
    return;
  }
  if (warp == 0) {
    tmem_alloc(&ctl->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int U = (int)(s_hi - s_lo);
  Cursor cur = s_cur;

  volatile int* abort_flag = &ctl->abort;
  // Each wait has its own limit (a long call may run for longer than one), set
  // only where the phase has not completed already.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = mbar_test_wait(bar, parity);
    if (!ok) ok = mbar_wait(bar, parity, abort_flag, global_timer_ns() + (uint64_t)p.timeout_ns);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = idesc_f16_f32(kRows, kKeys);
    constexpr uint32_t idesc_o = idesc_f16_f32(kRows, D) | (1u << 16);  // B is MN-major
    const uint64_t dq = sw128_desc(smem_u32(sQ));
    int s = 0, ph = 0, tq = 0, to = 0;  // ring place; tiles whose Q has been waited for, whose O has been started
    auto next_stage = [&]() {
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    };
    Cursor nxt = cur;                   // unit u + 1
    bool fresh = true;                  // unit u + 1 starts a tile (in this run)
    bool ok = true, ofresh = false;     // ofresh: unit u starts one
    for (int u = -1; ok && u < U; ++u) {
      bool nfresh = fresh;
      if (u + 1 < U) {
        // S of unit u + 1
        if (nfresh) ok = warp_wait(&ctl->q_full, tq++ & 1);
        const uint32_t d = tmem + kColS + 128 * ((u + 1) & 1);
        const bool ends = nxt.last() || u + 2 == U;
        for (int h = 0; ok && h < F::kKParts; ++h) {
          if (!warp_wait(&ctl->full[s], ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dk = sw128_desc(smem_u32(sR + s * F::kStageBytes));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < F::kKDims / 16; ++kk) {
              const uint32_t in = (kk >> 2) * (kKeys * 128 / 16) + (kk & 3) * 2;  // 64-dim slabs of 128 rows
              mma_f16(d, dq + (uint32_t)(h * (F::kKDims / 64)) * (kRows * 128 / 16) + in, dk + in, idesc_s, (h | kk) != 0);
            }
            mma_commit(&ctl->empty[s]);
            if (h == F::kKParts - 1) {
              mma_commit(&ctl->s_full[(u + 1) & 1]);
              if (ends) mma_commit(&ctl->q_empty);
            }
          }
          __syncwarp();
          next_stage();
        }
        fresh = nxt.last();
        if (u + 2 < U) nxt.advance(p, r);
      }
      if (ok && u >= 0) {
        // O of unit u
        ok = warp_wait(&ctl->p_full[u & 1], (u >> 1) & 1);
        if (ok && ofresh) {
          if (to > 0) ok = warp_wait(&ctl->o_empty, (to - 1) & 1);
          ++to;
        }
        const uint32_t a = tmem + kColS + 128 * (u & 1);
        for (int h = 0; ok && h < F::kVParts; ++h) {
          if (!warp_wait(&ctl->full[s], ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dv = sw128_mn_desc(smem_u32(sR + s * F::kStageBytes), F::kVKeys * 128);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < F::kVKeys / 16; ++kk)
              mma_f16_ta(tmem, a + (h * F::kVKeys + kk * 16) / 2, dv + kk * (16 * 128 / 16), idesc_o,
                         !(ofresh && h == 0 && kk == 0));
            mma_commit(&ctl->empty[s]);
            if (h == F::kVParts - 1) mma_commit(&ctl->pv_done[u & 1]);
          }
          __syncwarp();
          next_stage();
        }
      }
      ofresh = nfresh;
    }
    if (elect_one()) mma_commit(&ctl->mma_done);  // arrives once every issued MMA has finished
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // --------------------------------------------------------- softmax
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float m = kMinusBig, l = 0.f, rs = 0.f, sh = 0.f;
    int see = 0, tile = 0;
    bool fresh = true, mid = cur.i > 0;  // the tile's first unit in this run; the tile began in an earlier run
    bool ok = true;
    // scales of a unit's cache blocks: lane k holds those of the k-th 16 positions
    auto load_scales = [&](const Cursor& k, float& sk, float& sv) {
      const int pos = min(k.i * kKeys + 16 * (lane & 7), k.len - 1);
      const size_t at = (size_t)(k.b * p.Hkv + k.g) * p.nblk + (pos >> p.shift);
      sk = __ldg(p.ks + at);
      sv = __ldg(p.vs + at);
    };
    float sk, sv;
    load_scales(cur, sk, sv);
    for (int u = 0; u < U; ++u) {
      Cursor nxt = cur;
      float skn = 0.f, svn = 0.f;
      if (u + 1 < U) {
        nxt.advance(p, r);
        load_scales(nxt, skn, svn);
      }
      if (fresh) {
        if (!warp_wait(&ctl->rc_full[tile & 1], (tile >> 1) & 1)) {
          ok = false;
          break;
        }
        const RowConst& rc = ctl->rc[tile & 1];
        rs = rc.scale[row] * (kE4m3 ? 1.f : 16777216.f);
        sh = rc.shift[row];
        see = rc.see[row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->rc_empty[tile & 1]);
        m = kMinusBig;
        l = 0.f;
      }
      if (!warp_wait(&ctl->s_full[u & 1], (u >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t ts = lane_addr + kColS + 128 * (u & 1);
      const float svx = sv > 0.f ? sv : kScaleFloor;
      const float lsv = log2f(svx), rsv = 1.f / svx;
      const int left = see - cur.i * kKeys;  // visible positions from the unit's first on
      const bool masked = __any_sync(0xffffffffu, left < kKeys);
      // the unit's maximum
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[32];
        tmem_ld_32(ts + 32 * j, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = rs * __shfl_sync(0xffffffffu, sk, 2 * j + h);
          const float b = fmaf(a, sh, __shfl_sync(0xffffffffu, lsv, 2 * j + h));
          const uint64_t a2 = pack2(a, a), b2 = pack2(b, b);
          if (!masked) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 y = unpack2(fma2(pack2(x[16 * h + e], x[16 * h + e + 1]), a2, b2));
              mx = fmaxf(mx, fmaxf(y.x, y.y));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (32 * j + 16 * h + e < left) mx = fmaxf(mx, fmaf(x[16 * h + e], a, b));
          }
        }
      }
      const bool raise = mx > m + kSlack;
      if (fresh) {
        m = fmaxf(mx, kMinusBig);
      } else if (__any_sync(0xffffffffu, raise)) {
        // O and L to the new maximum, once the products of the last unit are in
        const float nm = raise ? mx : m, f = ex2(m - nm);
        m = nm;
        l *= f;
        if (!warp_wait(&ctl->pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int j = 0; j < D / 32; ++j) {
          float x[32];
          tmem_ld_32(lane_addr + 32 * j, x);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(x[16 * h + e] * f);
            tmem_st_16(lane_addr + 32 * j + 16 * h, w);
          }
        }
      }
      // weights, over S
      const float top = kWeightBits - m;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[32];
        tmem_ld_32(ts + 32 * j, x);
        uint32_t w[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = rs * __shfl_sync(0xffffffffu, sk, 2 * j + h);
          const float b = fmaf(a, sh, __shfl_sync(0xffffffffu, lsv, 2 * j + h)) + top;
          const float rv = __shfl_sync(0xffffffffu, rsv, 2 * j + h);
          const uint64_t a2 = pack2(a, a), b2 = pack2(b, b);
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float2 y = unpack2(fma2(pack2(x[16 * h + e], x[16 * h + e + 1]), a2, b2));
            if (masked) {
              y.x = 32 * j + 16 * h + e < left ? y.x : -INFINITY;
              y.y = 32 * j + 16 * h + e + 1 < left ? y.y : -INFINITY;
            }
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            s0 += y.x;
            s1 += y.y;
            w[8 * h + e / 2] = pack_f16(y.x, y.y);
          }
          l = fmaf(s0 + s1, rv, l);
        }
        tmem_st_16(ts + 16 * j, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[u & 1]);

      fresh = cur.last();
      if (cur.last() || u + 1 == U) {
        // ---- the run leaves this tile: its rows' outputs, or the partial state
        if (!warp_wait(&ctl->pv_done[u & 1], (u >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int rho = cur.rt * kRows + row;
        if (!mid && cur.last()) {
          const float inv = see > 0 ? 1.f / l : 0.f;
          const bool live = rho < cur.n * r && see > 0;
          uint16_t* orow = p.o + ((size_t)(cur.lo + (live ? rho / r : 0)) * p.Hq + (size_t)cur.g * r +
                                  (live ? rho % r : 0)) * D;
          for (int j = 0; j < D / 32; ++j) {
            float x[32];
            tmem_ld_32(lane_addr + 32 * j, x);
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const __nv_bfloat162 y = __floats2bfloat162_rn(x[e + 2 * k] * inv, x[e + 2 * k + 1] * inv);
                  w[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *reinterpret_cast<uint4*>(orow + 32 * j + e) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        } else {
          float* part = p.part + (size_t)(2 * c + (mid ? 0 : 1)) * slot_floats(D) + row;
          for (int j = 0; j < D / 32; ++j) {
            float x[32];
            tmem_ld_32(lane_addr + 32 * j, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) part[(size_t)(32 * j + e) * kRows] = x[e];
          }
          part[(size_t)D * kRows] = m;
          part[(size_t)(D + 1) * kRows] = l;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_empty);
        ++tile;
        mid = false;
        fresh = true;
      }
      cur = nxt;
      sk = skn;
      sv = svn;
    }
    (void)ok;
  } else if (warp >= 8) {
    // ---------------------------------------------- codes -> fp16 operands
    const int t = threadIdx.x - 256;
    constexpr int kKPieces = F::kKDims / 16, kVPieces = D / 16;  // 16-code pieces of a stage's row
    const int kpiece = t % kKPieces, kkey = t / kKPieces, vpiece = t % kVPieces, vkey = t / kVPieces;
    // Of the 8 lanes that store together, the upper 4 (the next 64-dim slab,
    // whose rows lie on the same banks) store their second chunk first.
    const int flip = D >= 128 ? (lane >> 2) & 1 : 0;
    struct Ref {  // a unit's codes
      size_t at;  // of its first position's first code
      int keys;   // positions that exist
    };
    auto ref = [&](const Cursor& k) -> Ref {
      return Ref{((size_t)(k.b * p.Hkv + k.g) * p.L_max + (size_t)k.i * kKeys) * D, k.len - k.i * kKeys};
    };
    auto load_k = [&](const Ref& f, int h, uint4 (&w)[F::kLoads]) {
#pragma unroll
      for (int i = 0; i < F::kLoads; ++i) {
        const int key = kkey + i * (kConvThreads / kKPieces);
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (key < f.keys) w[i] = ldg_nc_v4(p.codes[0] + f.at + (size_t)key * D + h * F::kKDims + kpiece * 16);
      }
    };
    auto load_v = [&](const Ref& f, int h, uint4 (&w)[F::kLoads]) {
#pragma unroll
      for (int i = 0; i < F::kLoads; ++i) {
        const int key = h * F::kVKeys + vkey + i * (kConvThreads / kVPieces);
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (key < f.keys) w[i] = ldg_nc_v4(p.codes[1] + f.at + (size_t)key * D + vpiece * 16);
        else if (!kE4m3) w[i] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
      }
    };
    auto store_piece = [&](uint32_t base, int rows, int key, int piece, const uint4& w, auto is_v) {
      constexpr bool kV = decltype(is_v)::value;
      uint32_t x[8];
      convert4<kE4m3, kV>(w.x, x[0], x[1]);
      convert4<kE4m3, kV>(w.y, x[2], x[3]);
      convert4<kE4m3, kV>(w.z, x[4], x[5]);
      convert4<kE4m3, kV>(w.w, x[6], x[7]);
      const uint32_t rowa = base + (uint32_t)(piece >> 2) * (rows * 128) + key * 128;
      const uint32_t ch = (uint32_t)(piece & 3) * 2, sw = key & 7;
      const uint32_t a0 = rowa + (((ch + flip) ^ sw) << 4), a1 = rowa + (((ch + (flip ^ 1)) ^ sw) << 4);
      if (flip) {
        sts128(a0, x[4], x[5], x[6], x[7]);
        sts128(a1, x[0], x[1], x[2], x[3]);
      } else {
        sts128(a0, x[0], x[1], x[2], x[3]);
        sts128(a1, x[4], x[5], x[6], x[7]);
      }
    };
    int s = 0, ph = 0, filled = 0;
    auto acquire = [&]() -> bool {
      if (filled >= kStages && !warp_wait(&ctl->empty[s], ph ^ 1)) return false;
      tc_fence_after();
      return true;
    };
    auto publish = [&]() {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->full[s]);
      ++filled;
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    };
    // Q of the tile at a cursor: two threads per row
    int tile = 0;
    auto load_q = [&](const Cursor& k) -> bool {
      if (tile > 0 && !warp_wait(&ctl->q_empty, (tile - 1) & 1)) return false;
      if (tile > 1 && !warp_wait(&ctl->rc_empty[tile & 1], ((tile >> 1) - 1) & 1)) return false;
      tc_fence_after();
      const int row = t >> 1, half = t & 1;
      const int rho = k.rt * kRows + row;
      const bool live = rho < k.n * r;
      const uint16_t* src = p.q + (size_t)(k.lo + (live ? rho / r : 0)) * p.q_stride +
                            (size_t)(k.g * r + (live ? rho % r : 0)) * D + half * (D / 2);
      uint32_t mx = 0u;
#pragma unroll 4
      for (int i = 0; i < D / 16; ++i) {
        const uint4 w = live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                   __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
      }
      mx = max(mx & 0xFFFFu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      const int e = min((int)(mx >> 7), 253);
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^-(e - 127)
      float sum = 0.f;
#pragma unroll 4
      for (int i = 0; i < D / 16; ++i) {
        const uint4 w = live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = pack_f16(bf16_bits_to_f32(in[j] & 0xFFFFu) * down, bf16_bits_to_f32(in[j] >> 16) * down);
          if (!kE4m3) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
            sum += y.x + y.y;
          }
        }
        const int d = half * (D / 2) + 8 * i;
        sts128(smem_u32(sQ) + (d >> 6) * (kRows * 128) + row * 128 + ((((d >> 3) & 7) ^ (row & 7)) << 4), x[0], x[1],
               x[2], x[3]);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      if (half == 0) {
        RowConst& rc = ctl->rc[tile & 1];
        rc.scale[row] = ldexpf(p.scale_log2, e - 127);
        rc.shift[row] = kE4m3 ? 0.f : sum * -7.62939453125e-06f;  // -128 2^-24
        rc.see[row] = live ? max(k.len - k.n + rho / r + 1, 0) : 0;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->q_full);
        mbar_arrive(&ctl->rc_full[tile & 1]);
      }
      ++tile;
      return true;
    };

    // Loads run two stages ahead of the stores. With two parts each of K and
    // V, buffer h holds part h: K of unit u + 1, then V of u, then K of u + 2;
    // with one part each, buffer 0 holds K and buffer 1 V.
    uint4 w0[F::kLoads], w1[F::kLoads];
    Cursor ck = cur;               // unit u + 1 (its Q)
    Cursor cn = cur;               // unit u + 2
    Ref f0 = ref(cur), f1 = f0;    // units u + 1 and u + 2 (f0 becomes unit u's when V comes)
    constexpr bool kTwo = F::kKParts == 2;
    load_k(f0, 0, w0);
    if (kTwo) load_k(f0, 1, w1);
    Ref fu = f0;                   // unit u
    bool ok = true, fresh = true;
    for (int u = -1; ok && u < U; ++u) {
      // here f0: unit u + 1, fu: unit u
      if (u + 2 < U) {
        cn.advance(p, r);
        f1 = ref(cn);
      }
      if (u + 1 < U) {
        if (fresh && !load_q(ck)) break;
        fresh = ck.last();
        if (!acquire()) break;
#pragma unroll
        for (int i = 0; i < F::kLoads; ++i)
          store_piece(smem_u32(sR + s * F::kStageBytes), kKeys, kkey + i * (kConvThreads / kKPieces), kpiece, w0[i],
                      std::false_type{});
        publish();
      }
      if (kTwo) {
        if (u >= 0) load_v(fu, 0, w0);
        if (u + 1 < U) {
          if (!acquire()) break;
#pragma unroll
          for (int i = 0; i < F::kLoads; ++i)
            store_piece(smem_u32(sR + s * F::kStageBytes), kKeys, kkey + i * (kConvThreads / kKPieces), kpiece, w1[i],
                        std::false_type{});
          publish();
        }
        if (u >= 0) {
          load_v(fu, 1, w1);
          if (!acquire()) break;
#pragma unroll
          for (int i = 0; i < F::kLoads; ++i)
            store_piece(smem_u32(sR + s * F::kStageBytes), F::kVKeys, vkey + i * (kConvThreads / kVPieces), vpiece,
                        w0[i], std::true_type{});
          publish();
        }
        if (u + 2 < U) load_k(f1, 0, w0);
        if (u >= 0) {
          if (!acquire()) break;
#pragma unroll
          for (int i = 0; i < F::kLoads; ++i)
            store_piece(smem_u32(sR + s * F::kStageBytes), F::kVKeys, vkey + i * (kConvThreads / kVPieces), vpiece,
                        w1[i], std::true_type{});
          publish();
        }
        if (u + 2 < U) load_k(f1, 1, w1);
      } else {
        if (u + 2 < U) load_k(f1, 0, w0);
        if (u >= 0) {
          if (!acquire()) break;
#pragma unroll
          for (int i = 0; i < F::kLoads; ++i)
            store_piece(smem_u32(sR + s * F::kStageBytes), F::kVKeys, vkey + i * (kConvThreads / kVPieces), vpiece,
                        w1[i], std::true_type{});
          publish();
        }
        if (u + 1 < U) load_v(f0, 0, w1);
      }
      fu = f0;
      f0 = f1;
      ck = cn;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    int dummy = 0;  // no MMA may still be running when TMEM is freed
    mbar_wait(&ctl->mma_done, 0, &dummy, global_timer_ns() + 100000000ull);
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0) p.flags[c] = *abort_flag ? (int32_t)MOE_ERR_DEVICE_TIMEOUT : 0;
}

struct MergeParams {
  const int32_t* offsets;
  const int32_t* lens;
  const float* part;
  const RunInfo* info;
  const int32_t* flags;
  uint16_t* o;
  int32_t* status;
  int Hq, Hkv, D, C;
};

constexpr int kMergeRows = 16;
constexpr int kMergeThreads = 256;

// Block (c, y): if run c is the second of the runs that share a tile, the
// tile's rows 16 y .. + 15. The first run of a tile left its state in its
// second slot (a tile that the run's end cuts), the others in their first.
__global__ void __launch_bounds__(kMergeThreads) kv8_tiles_merge_kernel(const MergeParams p) {
  __shared__ float s_f[kMaxCtas][kMergeRows];   // factor of each state and row
  __shared__ float s_o[kMergeRows][256 + 1];
  __shared__ int s_first;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, C = p.C, t = threadIdx.x;
  if (c == 0 && blockIdx.y == 0) {
    // the call's status: the outcome of the lowest-numbered grid block that failed
    if (t == 0) s_first = C;
    __syncthreads();
    for (int cc = t; cc < C; cc += kMergeThreads)
      if (__ldcg(p.flags + cc) != 0) atomicMin(&s_first, cc);
    __syncthreads();
    if (t == 0) *p.status = s_first == C ? 0 : __ldcg(p.flags + s_first);
  }
  const RunInfo f = p.info[c];
  if (!f.live || f.i == 0) return;
  const long long N = f.units, start = f.lo - f.i;
  const int c0 = cta_of(start, N, C);
  if (c != cta_of((long long)(c0 + 1) * N / C, N, C)) return;  // a later one of the tile's runs
  const int c1 = cta_of(start + f.nb - 1, N, C);
  const int r = p.Hq / p.Hkv, D = p.D, row0 = blockIdx.y * kMergeRows;
  const int lo = __ldg(p.offsets + f.b), n = __ldg(p.offsets + f.b + 1) - lo, len = __ldg(p.lens + f.b);
  const int row = t % kMergeRows;
  // every state's factor 2^(m_c - M) / L (empty runs have none)
  auto live = [&](int cc) { return (long long)cc * N / C != (long long)(cc + 1) * N / C; };
  auto slot = [&](int cc) { return p.part + (size_t)(2 * cc + (cc == c0 ? 1 : 0)) * slot_floats(D) + row0; };
  int failed = 0;
  for (int cc = c0 + t; cc <= c1; cc += kMergeThreads) failed |= live(cc) ? __ldcg(p.flags + cc) : 0;
  if (__syncthreads_or(failed)) return;  // a run gave up: o is left as it was
  if (t < kMergeRows) {
    float M = kMinusBig, L = 0.f;
    for (int cc = c0; cc <= c1; ++cc)
      if (live(cc)) M = fmaxf(M, __ldcg(slot(cc) + (size_t)D * kRows + t));
    for (int cc = c0; cc <= c1; ++cc) {
      const float e = live(cc) ? exp2f(__ldcg(slot(cc) + (size_t)D * kRows + t) - M) : 0.f;
      s_f[cc - c0][t] = e;
      if (live(cc)) L += e * __ldcg(slot(cc) + (size_t)(D + 1) * kRows + t);
    }
    const int rho = f.rt * kRows + row0 + t;
    const float inv = rho < n * r && len - n + rho / r >= 0 ? 1.f / L : 0.f;
    for (int cc = c0; cc <= c1; ++cc) s_f[cc - c0][t] *= inv;
  }
  __syncthreads();
  for (int d = t / kMergeRows; d < D; d += kMergeThreads / kMergeRows) {
    float acc = 0.f;
    for (int cc = c0; cc <= c1; ++cc)
      if (live(cc)) acc = fmaf(s_f[cc - c0][row], __ldcg(slot(cc) + (size_t)d * kRows + row), acc);
    s_o[row][d] = acc;
  }
  __syncthreads();
  for (int i = t; i < kMergeRows * D / 2; i += kMergeThreads) {
    const int rr = i / (D / 2), d = 2 * (i % (D / 2)), rho = f.rt * kRows + row0 + rr;
    if (rho >= n * r || len - n + rho / r < 0) continue;
    const __nv_bfloat162 y = __floats2bfloat162_rn(s_o[rr][d], s_o[rr][d + 1]);
    *reinterpret_cast<__nv_bfloat162*>(p.o + ((size_t)(lo + rho / r) * p.Hq + (size_t)f.g * r + rho % r) * D + d) = y;
  }
}

}  // namespace tiles

size_t tiles_workspace_bytes(const moe_kv8_shape& s) {
  using namespace tiles;
  return 256 + kMaxCtas * (sizeof(int32_t) + sizeof(RunInfo)) + 2 * kMaxCtas * slot_floats(s.D) * sizeof(float);
}

moe_status launch_tiles(const AttnArgs& a, cudaStream_t stream) {
  using namespace tiles;
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice, "device query");
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  int32_t* flags = reinterpret_cast<int32_t*>(ws + 256);
  RunInfo* info = reinterpret_cast<RunInfo*>(ws + 256 + kMaxCtas * sizeof(int32_t));
  float* part = reinterpret_cast<float*>(ws + 256 + kMaxCtas * (sizeof(int32_t) + sizeof(RunInfo)));
  const int shift = a.block == 16 ? 4 : a.block == 32 ? 5 : 6;
  const Params prm{a.q, {a.k, a.v}, a.ks, a.vs, a.offsets, a.lens, a.o, part, info, flags, a.scale_log2,
                   a.B, a.T, a.Hq, a.Hkv, a.L_max, a.nblk, shift, a.q_stride, kTimeoutNs};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto d, auto fp8) -> cudaError_t {
    constexpr int D = decltype(d)::value;
    constexpr bool kE4m3 = decltype(fp8)::value;
    static SmemLimitMemo smem_memo;
    const cudaError_t e = ensure_smem(kv8_tiles_kernel<D, kE4m3>, Cfg<D>::kBytes, &smem_memo);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = Cfg<D>::kBytes;
    return cudaLaunchKernelEx(&cfg, kv8_tiles_kernel<D, kE4m3>, prm);
  };
  auto pick = [&](auto fp8) {
    return a.D == 64    ? go(std::integral_constant<int, 64>{}, fp8)
           : a.D == 128 ? go(std::integral_constant<int, 128>{}, fp8)
                        : go(std::integral_constant<int, 256>{}, fp8);
  };
  cudaError_t e = a.e4m3 ? pick(std::true_type{}) : pick(std::false_type{});
  if (e != cudaSuccess) return cuda_fail(e, "tile kernel launch");
  const MergeParams mp{a.offsets, a.lens, part, info, flags, a.o, status, a.Hq, a.Hkv, a.D, grid};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)(kRows / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, kv8_tiles_merge_kernel, mp);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "merge kernel launch");
}

}  // namespace kv8
}  // namespace bgmoe
