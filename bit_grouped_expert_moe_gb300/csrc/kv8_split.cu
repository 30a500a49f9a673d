// Attention over the 8-bit KV cache for few query tokens per sequence
// (decode, verification of a few draft tokens), sm_103a.
//
// What bounds it is the cache's bytes: every position is read once per
// (sequence, KV head, row tile), where a row tile is 8 kNT rows and a row one
// (query token, query head of the KV head). The positions a tile can see are
// cut into units of 64 (D = 256) or 128 and all units of the call are laid end
// to end in the order (sequence, KV head, row tile, position) and dealt out in
// equal contiguous runs, one per block of a one-block-per-SM grid, so the bytes
// spread evenly over the SMs whatever the lengths are.
//
// Measured (16 heads on 2 x 256 but for the drafts, both kernels, in a run of calls):
//   one token after 131,072 positions, E4M3    30.6 us, 4.4 TB/s (65% of the
//                            measured copy rate; 7.6 us of it do not grow)
//   one token after 32,768 positions, INT8     14.8 us, 2.3 TB/s
//   a ragged batch of 8, 148,369 positions     34.0 us, 4.5 TB/s
//   1 to 5 drafts of 16 sequences, 70,120 positions, 4 x 128, E4M3   31.0 us,
//                            2.3 TB/s: 0.87 us a unit of 32 KB (0.74 at the copy
//                            rate), a fifth more of them than positions (second
//                            tiles, ragged ends), 3.3 us a tile begun and ended
// What does not grow (one token after 300 positions, from the wait for the
// predecessors): 1.6 us the tables and the run's start, 0.8 Q, 1.1 the first
// codes and their unit, 1.3 the fold, 0.9 to the merge's start, 1.5 the merge.
// A simple kernel, a block per row with plain loads, took 15.9 ms at 32,768
// positions.
//
// kv8_split_kernel — warp 8 streams each unit's K and V codes into a
// shared-memory ring by TMA. Four warps take 16 or 32 positions each;
// the other four take every second unit, or, where 8 kNT rows by D head dims
// are more than a warp's registers hold, the other half of the rows:
//   S^T  = K Q^T     mma.sync m16n8k16 in fp16: M = 16 positions, N = 8 rows;
//   online softmax per row on the base-2 scale;
//   O^T += V^T P^T   M = 16 head dims, N = 8 rows, K = 16 positions.
// Codes become fp16 operands in registers, after the ldmatrix:
//   int8 K  the byte u = code + 128 as an fp16 subnormal, u 2^-24 (one byte
//           permute per two values); the accumulators start at -128 sum(q) to
//           take the 128 out again;
//   int8 V  1024 + u by the same permute, minus 1152 (the sums over many
//           positions must not carry an offset that cancels in the end);
//   e4m3    the conversion instruction, exact in fp16.
// ldmatrix moves 16-bit units, so a transposed load of V leaves the two bytes
// of a unit, two neighbouring head dims, in one lane: they become rows g and
// g + 8 of the MMA (dims 2g and 2g + 1), a renaming of rows that only the
// store of O has to know. The same holds for the order of K's head dims
// within 16, which the Q fragments share.
//
// Scales: a warp's 16 positions lie in one cache block. K's scale multiplies
// the score. V's scale is folded into the softmax weight: with
//   x_j = score_j + log2 s_v(j),  w_j = 2^(x_j - m + 7),  m >= max x - 8,
// O = sum w_j code_j and L = sum w_j / s_v(j) give o = O / L. w <= 2^15 fits
// fp16, whose subnormals reach 2^-31 below a weight at m; L sums the
// fp32 weights, or what they stand for where those would vanish (kFar), so it
// also keeps blocks whose values are all zero (s_v taken as the smallest scale
// there). q goes to fp16 with its row's largest
// magnitude in [1, 2), an exact step apart from values 2^-14 and more below it.
//
// kv8_merge_kernel — one block per (query token, query head, 64 head dims)
// combines the partial states of the grid blocks that covered its tile, in a
// fixed order:
//   M = max m_c,  o = sum 2^(m_c - M) O_c / sum 2^(m_c - M) L_c.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <type_traits>

#include "kernels.h"
#include "kv8_attn.h"
#include "tc_ptx.cuh"

namespace bgmoe {
namespace kv8 {
namespace split {

using tc::elect_one;
using tc::mbar_arrive;
using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_test_wait;
using tc::mbar_wait;
using tc::smem_u32;

// Positions per unit (= ring stage): 16 per warp of four, 32 at the smaller head
// sizes, where two independent products hide one another's latency.
constexpr int unit_positions(int D) { return D == 256 ? 64 : 128; }
constexpr int kConsumers = 8;       // warps
// Three warpgroups, of which the third has one working warp: 9 warps would
// leave each thread 168 registers (three warps on one scheduler), so the third
// gives most of its own away: 256 x 232 + 128 x 40 = 384 x 168. (The consumers
// of 16 rows by 128 head dims spilled 45 words otherwise.)
constexpr int kThreads = (kConsumers + 4) * 32;
constexpr int kLaunchRegs = 168, kConsumerRegs = 232, kProducerRegs = 40;
static_assert(kConsumers * kConsumerRegs + 4 * kProducerRegs <= (kConsumers + 4) * kLaunchRegs &&
                  kConsumerRegs >= kLaunchRegs && kProducerRegs <= kLaunchRegs,
              "register shares");
constexpr int kMaxCtas = 256;       // workspace bound on the grid
// Beginning and ending a tile (Q, the warps' fold, the partial state) costs a
// run about as much as four units: 3 us against 0.7 us a unit of 32 KB. A
// ragged batch of 8 takes 37.9, 33.4, 32.9 us at 2, 4 and 6, the drafts of 16
// sequences 34.0, 33.3, 34.3.
constexpr int kTileCost = 4;
constexpr float kMinusBig = -3.402823466e38f;  // running-max start, finite: 2^(m - m_new) is never NaN
// A row's m is raised to its largest score only when a score passes it by
// more than kSlack: weights are 2^kWeightBits at m and fit fp16 up to there.
// From 2^23 on, where an fp32 step is 1 and more and m + 8 or m - 7 may be
// rounded away from each other, whenever a score passes it.
constexpr float kWeightBits = 7.f, kSlack = 8.f;

template <int D, int kNT>
struct Cfg {
  static constexpr int kRowSplit = kNT * D > 256 ? 2 : 1;  // warps that share positions and split the rows
  static constexpr int kNTw = kNT / kRowSplit;             // groups of 8 rows of a warp
  static constexpr int kFold = kConsumers / kRowSplit;     // warps whose states belong to the same rows
  static constexpr int kUsers = kRowSplit == 2 ? 8 : 4;    // warps that read a unit
  static constexpr int kStride = kRowSplit == 2 ? 1 : 2;   // from one unit of a warp to its next
  static constexpr int kSlabs = D < 128 ? 1 : D / 128;    // TMA boxes of up to 128 bytes by kPos rows
  static constexpr int kPos = unit_positions(D);
  static constexpr int kMT = kPos / 64;                    // products of 16 positions of a warp
  static constexpr int kSlab = kPos * (D < 128 ? D : 128);
  static constexpr int kStageBytes = 2 * kSlabs * kSlab;  // K then V
  static constexpr int kFoldItems = kNTw * (D / 16) * 32;  // a warp's accumulators, four at a time
  static constexpr int kFoldBytes = 4 * kFoldItems * 16;   // four slots
  static constexpr int kQPitch = D * 2 + 32;              // bytes of a row of Q (the padding spreads the banks)
  static constexpr int kQBytes = 8 * kNT * kQPitch;
  static constexpr int kFit = (223 * 1024 - kFoldBytes - kQBytes) / kStageBytes;
  // an even number: the warps that take every second unit have stages of their own
  static constexpr int kStages = kFit > 12 ? 12 : kFit & ~1;
  static constexpr int kFoldOffset = kStages * kStageBytes;
  static constexpr int kQOffset = kFoldOffset + kFoldBytes;
  static constexpr int kCtlOffset = kQOffset + kQBytes;
  static constexpr int kBytes = kCtlOffset + 2816 + 1024;  // + alignment slack
  static_assert(kNTw * D <= 256 && kStages >= 3 && kBytes <= 227 * 1024, "registers and shared memory");
};

template <int kStages>
struct Ctl {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t fold;  // all consumer warps, at each step of a fold
  uint64_t go;    // all consumer warps have asked for their first tile's Q and scales
  int abort;
  // of the tile's rows: score factor of the row's power of two, -128 sum(q)
  // 2^-24 (int8), visible positions
  float scale[32], shift[32];
  int see[32];
  float m[kConsumers][32], l[kConsumers][32];  // the warps' states, at a fold
};

struct Params {
  const uint16_t* q;
  const float* ks;
  const float* vs;
  const int32_t* offsets;
  const int32_t* lens;
  float* part;       // [slots][RT] m, then [slots][RT] l, then [slots][RT][D] O
  int4* info;        // [C]: the tile and unit a block's run starts at: {tile, has units, unit}
  int32_t* flags;    // [C]: every grid block's outcome (0 or a moe_status), written each call
  long long slots;
  float scale_log2;
  int B, T, Hq, Hkv, L_max, nblk, shift, q_stride;  // shift: log2 of the cache's block
  int stalled;
  long long timeout_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// d += A * B, A 16x16 (row), B 16x8 (col), fp16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

// Bytes 0, 1 and bytes 2, 3 of a K word as fp16 pairs (int8: u 2^-24).
template <bool kE4m3>
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (kE4m3) {
    p01 = e4m3x2_f16x2(w);
    p23 = e4m3x2_f16x2(w >> 16);
  } else {
    p01 = __byte_perm(w, 0u, 0x4140);
    p23 = __byte_perm(w, 0u, 0x4342);
  }
}

// Bytes 0, 2 and bytes 1, 3 of a V word as fp16 pairs (int8: the code).
template <bool kE4m3>
__device__ __forceinline__ void v_pairs(uint32_t w, uint32_t& p02, uint32_t& p13) {
  if (kE4m3) {
    const uint32_t x = __byte_perm(w, 0u, 0x3120);
    p02 = e4m3x2_f16x2(x);
    p13 = e4m3x2_f16x2(x >> 16);
  } else {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4240), b = __byte_perm(w, 0x64646464u, 0x4341);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    p02 = *reinterpret_cast<const uint32_t*>(&x);
    p13 = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Place in the run: unit i of the nb units of row tile rt of KV head g of
// sequence b; `tile` numbers the row tiles of the call.
struct Cursor {
  int b, g, rt, i, nb, n, len, lo, tile;
  __device__ void sequence(const Params& p) {  // tables of sequence b (b < B)
    lo = ld(p.offsets + b);
    n = ld(p.offsets + b + 1) - lo;
    len = ld(p.lens + b);
  }
  // The next unit; the caller knows that there is one.
  __device__ void advance(const Params& p, int r, int RT, int kPos) {
    if (++i < nb) return;
    i = 0;
    do {
      ++tile;
      if (++rt >= seq_tiles(n, r, RT)) {
        rt = 0;
        if (++g >= p.Hkv) {
          g = 0;
          do {
            if (++b >= p.B) return;
            sequence(p);
          } while (n == 0);
        }
      }
      nb = tile_units(n, len, r, RT, kPos, rt);
    } while (nb == 0);
  }
};

template <int D, int kNT, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const Params p) {
  using S = Cfg<D, kNT>;
  constexpr int kNTw = S::kNTw, kPos = S::kPos, kMT = S::kMT;
  constexpr int kStages = S::kStages;
  constexpr int RT = 8 * kNT;  // rows of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl<kStages>* ctl = reinterpret_cast<Ctl<kStages>*>(smem + S::kCtlOffset);
  static_assert(sizeof(Ctl<kStages>) <= 2816, "control block");
  float* mrg = reinterpret_cast<float*>(smem + S::kFoldOffset);
  __shared__ long long s_unit[2];  // units before the run's start and end
  __shared__ Cursor s_cur;
  __shared__ int s_bad;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = gridDim.x, c = blockIdx.x;
  const int r = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], S::kUsers);
    }
    mbar_init(&ctl->fold, kConsumers);
    mbar_init(&ctl->go, kConsumers);
    ctl->abort = 0;
    tc::fence_barrier_init();
  }
  if (warp == kConsumers) {
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  // Launched with programmatic dependent launch: the setup above overlaps the
  // previous kernel on the stream. Everything below may read what earlier
  // kernels wrote or overwrite what they read (the partial states and flags),
  // so it waits for them first. Only then may this call's merge launch: it
  // reads the tables before its own wait.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 2) {  // the run's start and its end
    Place k;
    const bool ok = find_run(p.offsets, p.lens, p.B, p.T, p.Hkv, p.L_max, r, RT, kPos, kTileCost, c + warp, C, &k);
    if (lane == 0) {
      s_unit[warp] = k.units;
      if (warp == 0) {
        s_bad = !ok;
        Cursor cur{};
        if (ok && k.b >= 0) {
          cur.b = k.b;
          cur.lo = k.lo;
          cur.n = k.n;
          cur.len = k.len;
          cur.g = k.g;
          cur.rt = k.rt;
          cur.i = k.i;
          cur.nb = k.nb;
          cur.tile = k.tile;
        }
        s_cur = cur;
      }
    }
  }
  __syncthreads();
  const bool live = !s_bad && s_unit[0] < s_unit[1];
  if (threadIdx.x == 0) {
    p.info[c] = make_int4(s_cur.tile, live, s_cur.i, 0);
    if (!live) p.flags[c] = s_bad ? (int32_t)MOE_ERR_INVALID_ARG : 0;
  }
  if (!live) return;
  const int U = (int)(s_unit[1] - s_unit[0]);
  Cursor cur = s_cur;

  volatile int* abort_flag = &ctl->abort;
  // Each wait has its own limit (a long call may run for longer than one), set
  // only where the phase has not completed already.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = mbar_test_wait(bar, parity);
    if (!ok) ok = mbar_wait(bar, parity, abort_flag, global_timer_ns() + (uint64_t)p.timeout_ns);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp >= kConsumers) {
    fewer_registers<kProducerRegs>();
    // ------------------------------------------------------------ producer
    if (warp == kConsumers) {
      // The first tile's Q and scales ask first: behind a ring's worth of codes
      // from every SM they took 3 us more.
      int s = 0, ph = 0, issued = 0;
      bool go = c != p.stalled && warp_wait(&ctl->go, 0);
#pragma unroll 1
      for (int j = 0; go && j < U; ++j) {
        if (issued >= kStages && !warp_wait(&ctl->empty[s], ph ^ 1)) break;
        if (elect_one()) {
          uint8_t* st = smem + s * S::kStageBytes;
          const int pair = cur.b * p.Hkv + cur.g;
          mbar_arrive_expect_tx(&ctl->full[s], (uint32_t)S::kStageBytes);
#pragma unroll
          for (int sl = 0; sl < S::kSlabs; ++sl) {
            tma_load_3d(st + sl * S::kSlab, &tm_k, sl * 128, cur.i * kPos, pair, &ctl->full[s]);
            tma_load_3d(st + (S::kSlabs + sl) * S::kSlab, &tm_v, sl * 128, cur.i * kPos, pair, &ctl->full[s]);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
        cur.advance(p, r, RT, kPos);
      }
      if (lane == 0 && *abort_flag) {  // let this block's own copies land before it exits
        int dummy = 0;
        const uint64_t dl = global_timer_ns() + 100000000ull;
        for (int k = issued - kStages < 0 ? 0 : issued - kStages; k < issued; ++k)
          mbar_wait(&ctl->full[k % kStages], (k / kStages) & 1, &dummy, dl);
      }
    }
  } else {
    // ----------------------------------------------------------- consumers
    more_registers<kConsumerRegs>();
    const int gq = lane >> 2, m4 = lane & 3;
    // ldmatrix row addresses (relative to a slab): lanes 0-7, 8-15, 16-23,
    // 24-31 address the four 8 x 16-byte matrices (positions +0, +8 of the
    // low 16 dims, then of the high 16)
    const int pw = warp & 3, part = warp >> 2;  // the warp's 16 kMT positions; its half of the units or of the rows
    const int rows0 = S::kRowSplit == 2 ? part * 8 * kNTw : 0;
    const int row = 16 * kMT * pw + (lane & 7) + ((lane >> 3) & 1) * 8;
    const int ch = lane >> 4;
    // TMA swizzle: 16-byte chunk ^= row % 8 (128-byte rows), (row / 2) % 4 (64-byte rows)
    constexpr int kRowBytes = D < 128 ? 64 : 128;
    const int sw = D < 128 ? (row >> 1) & 3 : row & 7;

    uint32_t qf[kNTw][D / 16][2];   // Q as the B operand: row 8 nt + gq, dims 16 ks + 4 m4 .. + 3
    float acc[kNTw][D / 16][4];
    float m[kNTw][2], l[kNTw][2];    // of rows 8 nt + 2 m4, + 1
    float rq[kNTw][2], off[kNTw][2]; // score factor of the row's power of two; -128 sum(q) 2^-24 (int8)
    int lim[kNTw][2];                // visible positions
    float top_sv = 0.f;              // the largest V scale of the tile's units so far
    int folds = 0;
    // All consumer warps have come this far.
    auto together = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->fold);
      return warp_wait(&ctl->fold, folds++ & 1);
    };
    // Q of a tile: a warp asks for one row at a time (fetch_q), converts it into
    // shared memory and every warp takes its fragments from there (place_q).
    // (Each warp fetching its own fragments took 4.7 us, at every tile: three
    // times the instructions, all of them cold.)
    constexpr int kPer = D / 32;  // head dims of a lane
    uint32_t raw[kNT][kPer / 2];
    auto fetch_q = [&](const Cursor& k) {
#pragma unroll
      for (int i = 0; i < kNT; ++i) {
        const int rr = k.rt * RT + warp + 8 * i, tok = rr / r;
        const bool live = rr < k.n * r;
        const uint16_t* src = p.q + (size_t)(k.lo + (live ? tok : 0)) * p.q_stride +
                              (size_t)(k.g * r + (live ? rr - tok * r : 0)) * D + kPer * lane;
        if constexpr (kPer == 8)
          asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(raw[i][0]), "=r"(raw[i][1]), "=r"(raw[i][2]), "=r"(raw[i][3])
                       : "l"(src)
                       : "memory");
        else if constexpr (kPer == 4)
          asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(raw[i][0]), "=r"(raw[i][1]) : "l"(src) : "memory");
        else
          asm volatile("ld.global.b32 %0, [%1];" : "=r"(raw[i][0]) : "l"(src) : "memory");
      }
    };
    const uint32_t sQ = smem_u32(smem + S::kQOffset);
    auto place_q = [&](const Cursor& t) -> bool {
#pragma unroll
      for (int i = 0; i < kNT; ++i) {
        const int rw = warp + 8 * i, rr = t.rt * RT + rw;
        const bool live = rr < t.n * r;
        uint32_t mx = 0u;
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          raw[i][k] = live ? raw[i][k] : 0u;
          mx = __vmaxu2(mx, raw[i][k] & 0x7FFF7FFFu);
        }
        mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
        // 2^-e with e the exponent of the largest magnitude (an infinity or a
        // NaN makes the whole row NaN whatever e is)
        const int e = min((int)(mx >> 7), 253);
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        float sum = 0.f;
        const uint32_t to = sQ + rw * S::kQPitch + 2 * kPer * lane;
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          const uint32_t x = pack_f16(__uint_as_float(raw[i][k] << 16) * down,
                                      __uint_as_float(raw[i][k] & 0xFFFF0000u) * down);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x));
          sum += a.x + a.y;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 4 * k), "r"(x) : "memory");
        }
        if (!kE4m3) {
#pragma unroll 1
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane == 0) {
          ctl->scale[rw] = p.scale_log2 * __uint_as_float(e > 0 ? (uint32_t)e << 23 : 0x00400000u);  // 2^(e - 127)
          ctl->shift[rw] = kE4m3 ? 0.f : sum * -7.62939453125e-06f;  // -128 2^-24
          ctl->see[rw] = live ? t.len - t.n + rr / r + 1 : 0;
        }
      }
      if (!together()) return false;
      top_sv = 0.f;
#pragma unroll
      for (int nt = 0; nt < kNTw; ++nt) {
        const uint32_t at = sQ + (rows0 + 8 * nt + gq) * S::kQPitch + 8 * m4;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(qf[nt][ks][0]), "=r"(qf[nt][ks][1])
                       : "r"(at + 32 * ks)
                       : "memory");
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int rw = rows0 + 8 * nt + 2 * m4 + k;
          rq[nt][k] = ctl->scale[rw];
          off[nt][k] = ctl->shift[rw];
          lim[nt][k] = ctl->see[rw];
          m[nt][k] = kMinusBig;
          l[nt][k] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) acc[nt][mt][0] = acc[nt][mt][1] = acc[nt][mt][2] = acc[nt][mt][3] = 0.f;
      }
      return true;
    };
    // The scales of this warp's positions of the unit at a cursor, 16 at a time
    // (a group past the context repeats the last position's: it is not used).
    auto load_scales = [&](const Cursor& k, float (&sk)[kMT], float (&sv)[kMT]) {
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        const int pos = min(k.i * kPos + 16 * (kMT * pw + t), k.len - 1);
        const size_t at = (size_t)(k.b * p.Hkv + k.g) * p.nblk + (pos >> p.shift);
        sk[t] = ld(p.ks + at);
        sv[t] = ld(p.vs + at);
      }
    };
    float skn[kMT], svn[kMT];  // of the next unit that is this warp's
    fetch_q(cur);
    {
      Cursor own = cur;
      if (S::kRowSplit == 1 && part == 1 && U > 1) own.advance(p, r, RT, kPos);
      load_scales(own, skn, svn);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->go);
    bool good = place_q(cur);

    int s = 0, ph = 0;
#pragma unroll 1
    for (int j = 0; good && j < U; ++j) {
      Cursor nxt = cur;
      if (j + 1 < U) {
        nxt.advance(p, r, RT, kPos);
        if (nxt.tile != cur.tile) fetch_q(nxt);  // it travels while this unit is computed
      }
      const bool mine = S::kRowSplit == 2 || (j & 1) == part;
      float sk[kMT], sv[kMT];
      if (mine) {
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          sk[t] = skn[t];
          sv[t] = svn[t];
        }
        if (j + S::kStride < U) {  // the scales of this warp's next unit travel, too
          Cursor own = nxt;
          if (S::kStride == 2) own.advance(p, r, RT, kPos);
          load_scales(own, skn, svn);
        }
        if (!warp_wait(&ctl->full[s], ph)) break;
      }
      const uint32_t sK = smem_u32(smem + s * S::kStageBytes);
      const uint32_t sV = sK + S::kSlabs * S::kSlab;
      auto chunk_addr = [&](uint32_t base, int kk, int t) -> uint32_t {  // dims 32 kk .. + 31 of the t-th 16 positions
        constexpr int kPerSlab = D < 128 ? 2 : 4;
        const int cc = (kk % kPerSlab) * 2 + ch;
        return base + (kk / kPerSlab) * S::kSlab + (row + 16 * t) * kRowBytes + ((cc ^ sw) << 4);
      };
      const int pos0 = cur.i * kPos + 16 * kMT * pw;  // this warp's first position
      if (mine && pos0 < cur.len) {
        float x[kMT][kNTw][4];
        float y[4] = {0.f, 0.f, 0.f, 0.f};  // one product: a second accumulator halves the dependent chain
        constexpr bool kHalve = kNTw * kMT == 1;
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt) {
            x[t][nt][0] = x[t][nt][2] = off[nt][0];
            x[t][nt][1] = x[t][nt][3] = off[nt][1];
          }
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
          for (int t = 0; t < kMT; ++t) {
            uint32_t w[4], a0, a1, a2, a3;
            ldsm_x4(chunk_addr(sK, kk, t), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              k_pairs<kE4m3>(w[2 * h], a0, a2);
              k_pairs<kE4m3>(w[2 * h + 1], a1, a3);
#pragma unroll
              for (int nt = 0; nt < kNTw; ++nt) {
                if (kHalve && h == 1) mma_f16(y, a0, a1, a2, a3, qf[nt][2 * kk + h][0], qf[nt][2 * kk + h][1]);
                else mma_f16(x[t][nt], a0, a1, a2, a3, qf[nt][2 * kk + h][0], qf[nt][2 * kk + h][1]);
              }
            }
          }
        // scores, with V's scale; does one pass its row's m by more than the slack?
        float rsv[kMT], bar[kNTw][2];
        bool up = false, far = false;
#pragma unroll
        for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) bar[nt][k] = fabsf(m[nt][k]) < 8388608.f ? m[nt][k] + kSlack : m[nt][k];
#pragma unroll
        for (int t = 0; t < kMT; ++t) top_sv = fmaxf(top_sv, sv[t]);
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          const float svx = sv[t] > 0.f ? sv[t] : kScaleFloor;
          const float lsv = __log2f(svx);
          rsv[t] = __fdividef(1.f, svx);
          far |= svx < kFar * top_sv;
          const int pr = pos0 + 16 * t + gq;
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float d = x[t][nt][e];
              if (kHalve) d += y[e];
              if (!kE4m3) d *= 16777216.f;
              x[t][nt][e] = pr + (e >> 1) * 8 < lim[nt][e & 1] ? fmaf(d, rq[nt][e & 1] * sk[t], lsv) : -INFINITY;
              up |= x[t][nt][e] > bar[nt][e & 1];
            }
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt) {
            float al[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float mx = m[nt][k];
#pragma unroll
              for (int t = 0; t < kMT; ++t) mx = fmaxf(mx, fmaxf(x[t][nt][k], x[t][nt][k + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const float root = ex2(0.5f * (m[nt][k] - mx));
              al[k] = root * root;
              m[nt][k] = mx;
              l[nt][k] = l[nt][k] * root * root;
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              acc[nt][mt][0] *= al[0];
              acc[nt][mt][1] *= al[1];
              acc[nt][mt][2] *= al[0];
              acc[nt][mt][3] *= al[1];
            }
          }
        }
        if (far) {  // the whole warp alike
#pragma unroll
          for (int t = 0; t < kMT; ++t) {
            const float svx = sv[t] > 0.f ? sv[t] : kScaleFloor;
            if (svx < kFar * top_sv) {
              const float lift = kLiftBits - __log2f(svx);
#pragma unroll
              for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float mk = m[nt][k] - kWeightBits;
                  l[nt][k] = fmaf(ex2(x[t][nt][k] - mk + lift) + ex2(x[t][nt][k + 2] - mk + lift), kUnlift, l[nt][k]);
                }
              rsv[t] = 0.f;
            }
          }
        }
        // weights; P^T as the B operand: rows (k) = positions, columns (n) = query rows
        uint32_t pb[kMT][kNTw][2];
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(x[t][nt][e] - (m[nt][e & 1] - kWeightBits));
#pragma unroll
            for (int k = 0; k < 2; ++k) l[nt][k] = fmaf(w[k] + w[k + 2], rsv[t], l[nt][k]);
            pb[t][nt][0] = movmatrix_trans(pack_f16(w[0], w[1]));
            pb[t][nt][1] = movmatrix_trans(pack_f16(w[2], w[3]));
          }
        // V bytes past the context may hold anything, a NaN of e4m3 included: zero them
        const bool tail = pos0 + 16 * kMT > cur.len;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
          for (int t = 0; t < kMT; ++t) {
            uint32_t w[4], a0, a1, a2, a3;
            ldsm_x4_trans(chunk_addr(sV, kk, t), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              v_pairs<kE4m3>(w[2 * h], a0, a1);      // positions 0-7: dims 2g, 2g + 1
              v_pairs<kE4m3>(w[2 * h + 1], a2, a3);  // positions 8-15
              if (kE4m3 && tail) {
                const int kp = pos0 + 16 * t + 2 * m4;
                const uint32_t mlo = (kp < cur.len ? 0x0000FFFFu : 0u) | (kp + 1 < cur.len ? 0xFFFF0000u : 0u);
                const uint32_t mhi = (kp + 8 < cur.len ? 0x0000FFFFu : 0u) | (kp + 9 < cur.len ? 0xFFFF0000u : 0u);
                a0 &= mlo;
                a1 &= mlo;
                a2 &= mhi;
                a3 &= mhi;
              }
#pragma unroll
              for (int nt = 0; nt < kNTw; ++nt)
                mma_f16(acc[nt][2 * kk + h], a0, a1, a2, a3, pb[t][nt][0], pb[t][nt][1]);
            }
          }
      }
      __syncwarp();
      if (mine && lane == 0) mbar_arrive(&ctl->empty[s]);
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }

      if (nxt.tile != cur.tile || j == U - 1) {
        // ---- the run leaves this tile: fold the states of the warps with the
        // same rows. All take the largest m; then, lane by lane, the upper half
        // of the warps hands its accumulators to the lower, and every thread
        // sums a part of what is left (a fixed order).
        const int idx = S::kRowSplit == 2 ? pw : warp, set0 = warp - idx;  // set0: the first warp of these rows
#pragma unroll
        for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], o);
            if (lane < 4) ctl->m[warp][8 * nt + 2 * lane + k] = m[nt][k];
          }
        if (!together()) break;
#pragma unroll
        for (int nt = 0; nt < kNTw; ++nt) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = m[nt][k];
#pragma unroll
            for (int w = 0; w < S::kFold; ++w) top = fmaxf(top, ctl->m[set0 + w][8 * nt + 2 * m4 + k]);
            const float root = ex2(0.5f * (m[nt][k] - top));
            f[k] = root * root;
            m[nt][k] = top;
            if (lane < 4) ctl->l[warp][8 * nt + 2 * lane + k] = l[nt][k] * root * root;
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            acc[nt][mt][0] *= f[0];
            acc[nt][mt][1] *= f[1];
            acc[nt][mt][2] *= f[0];
            acc[nt][mt][3] *= f[1];
          }
        }
        constexpr int kHalf = S::kFold / 2;  // slots of a set of rows
        float4* slots = reinterpret_cast<float4*>(smem + S::kFoldOffset);
        float4* own = slots + (set0 / 2 + (idx < kHalf ? idx : idx - kHalf)) * S::kFoldItems + lane;
        if (idx >= kHalf) {
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
              own[(nt * (D / 16) + mt) * 32] =
                  make_float4(acc[nt][mt][0], acc[nt][mt][1], acc[nt][mt][2], acc[nt][mt][3]);
        }
        if (!together()) break;
        if (idx < kHalf) {
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              const float4 o = own[(nt * (D / 16) + mt) * 32];
              own[(nt * (D / 16) + mt) * 32] = make_float4(acc[nt][mt][0] + o.x, acc[nt][mt][1] + o.y,
                                                           acc[nt][mt][2] + o.z, acc[nt][mt][3] + o.w);
            }
        }
        if (!together()) break;
        const size_t slot = (size_t)c + cur.tile;
        float* po = p.part + (size_t)2 * p.slots * RT + slot * RT * D;
#pragma unroll
        for (int it = 0; it < S::kRowSplit * S::kFoldItems; it += kConsumers * 32) {
          const int item = it + warp * 32 + lane, set = item / S::kFoldItems, in = item % S::kFoldItems;
          if (item >= S::kRowSplit * S::kFoldItems) break;
          float4 o = slots[set * kHalf * S::kFoldItems + in];
#pragma unroll
          for (int w = 1; w < kHalf; ++w) {
            const float4 a = slots[(set * kHalf + w) * S::kFoldItems + in];
            o = make_float4(o.x + a.x, o.y + a.y, o.z + a.z, o.w + a.w);
          }
          const int ln = in & 31, nt = (in >> 5) / (D / 16), mt = (in >> 5) % (D / 16);
          float* at = po + (size_t)(set * 8 * kNTw + 8 * nt + 2 * (ln & 3)) * D + 16 * mt + 2 * (ln >> 2);
          *reinterpret_cast<float2*>(at) = make_float2(o.x, o.z);
          *reinterpret_cast<float2*>(at + D) = make_float2(o.y, o.w);
        }
        if (idx == 0 && lane < 8 * kNTw) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < S::kFold; ++w) sum += ctl->l[set0 + w][lane];
          p.part[(size_t)p.slots * RT + slot * RT + rows0 + lane] = sum;
        }
        if (idx == 0 && lane < 4) {
#pragma unroll
          for (int nt = 0; nt < kNTw; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) p.part[slot * RT + rows0 + 8 * nt + 2 * lane + k] = m[nt][k];
        }
        cur = nxt;
        if (j + 1 < U) good = place_q(cur);
      } else {
        cur = nxt;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.flags[c] = *abort_flag ? (int32_t)MOE_ERR_DEVICE_TIMEOUT : 0;
}

struct MergeParams {
  const int32_t* offsets;
  const int32_t* lens;
  const float* part;
  const int4* info;
  const int32_t* flags;
  uint16_t* o;
  int32_t* status;
  long long slots;
  int B, T, Hq, Hkv, D, L_max, RT, C;
};

// Thread t holds dims 4 (t % 16) .. + 3 of the slice and takes the covering grid
// blocks c0 + t / 16, c0 + kLanes + t / 16, ...: all loads of kMergeBatch states
// are issued before any is used. Then the kLanes sums are merged in shared memory.
// 16 of them, or 4 where the SMs do not hold that many threads for every row and
// slice at once (many rows have few states each): see launch_split.
constexpr int kMergeBatch = 5;  // 16 times 5: the 76 states of a pair of two on 152 SMs at once

template <int kLanes>
__global__ void __launch_bounds__(kLanes * 16) kv8_merge_kernel(const MergeParams p) {
  constexpr int kMergeWarps = kLanes / 2;
  // The next call's split kernel may launch now: it waits for this grid to
  // finish before it touches the workspace.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Everything up to the dependency wait reads only the tables, which the
  // split kernel does not write: it overlaps that kernel's tail. Whatever wrote
  // them ended before the split kernel let this one launch, so L2 has them; L1,
  // which nobody invalidates before the wait, is not asked. One warp of a block
  // asks: where both did, a token of 64 sequences of 2000 positions took 41.3 us for
  // 38.5.
  const int r = p.Hq / p.Hkv, RT = p.RT, C = p.C, D = p.D;
  const int t = blockIdx.x / p.Hq, h = blockIdx.x - t * p.Hq;
  const int lane = threadIdx.x & 31, f4 = threadIdx.x & 15, sl = threadIdx.x >> 4;
  __shared__ float s_m[kLanes], s_l[kLanes], s_o[kLanes][64];
  __shared__ int s_range[2], s_first, s_tiles, s_b;
  __shared__ int3 s_seq;
  if (threadIdx.x < 32) {  // the sequence, and the tiles before it
    int tiles = 0, b = -1;
    int3 seq = make_int3(0, 0, 0);
    bool bad = false;
#pragma unroll 1
    for (int base = 0; base < p.B; base += 32) {
      const int bb = base + lane;
      int lo1 = 0, hi1 = 0, len1 = 0;
      if (bb < p.B) {
        lo1 = __ldcg(p.offsets + bb);
        hi1 = __ldcg(p.offsets + bb + 1);
        len1 = __ldcg(p.lens + bb);
        bad |= offsets_bad(lo1, hi1, bb, p.B, p.T) || len1 < 0 || len1 > p.L_max;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, lo1 <= t && t < hi1);
      tiles += __reduce_add_sync(0xffffffffu, hi1 <= t ? seq_tiles(hi1 - lo1, r, RT) : 0);
      if (hit) {
        const int L = __ffs(hit) - 1;
        b = base + L;
        seq.x = __shfl_sync(0xffffffffu, lo1, L);
        seq.y = __shfl_sync(0xffffffffu, hi1 - lo1, L);
        seq.z = __shfl_sync(0xffffffffu, len1, L);
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s_tiles = tiles;
      s_b = bad ? -1 : b;
      s_seq = seq;
      s_range[0] = s_range[1] = -1;
      s_first = C;
    }
  }
  __syncthreads();
  const bool bad = s_b < 0;
  const int lo = s_seq.x, n = s_seq.y, len = s_seq.z;
  const int g = h / r, row = (t - lo) * r + h - g * r, rt = row / RT;
  const int tile = bad ? 0 : s_tiles * p.Hkv + g * seq_tiles(n, r, RT) + rt;
  const size_t slot0 = bad ? 0 : (size_t)tile * RT + row - rt * RT;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The runs that cover the tile: from the last one that starts at or before
  // its first unit to the last one that starts in it. And the call's status:
  // the outcome of the lowest-numbered grid block that failed.
#pragma unroll 1
  for (int cc = threadIdx.x; cc < C; cc += kMergeWarps * 32) {
    const int4 x = __ldcg(p.info + cc);
    if (__ldcg(p.flags + cc) != 0) atomicMin(&s_first, cc);
    if (x.y && x.x <= tile) {
      atomicMax(&s_range[1], cc);
      if (x.x < tile || x.z == 0) atomicMax(&s_range[0], cc);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *p.status = s_first == C ? 0 : __ldcg(p.flags + s_first);
  const bool seen = len - n + (t - lo) >= 0;  // else no visible position
  const int c0 = seen ? s_range[0] : 0, c1 = seen ? s_range[1] : -1;
  if (bad) return;

  const float* pm = p.part;
  const float* pl = p.part + (size_t)p.slots * RT;
  const float* po = p.part + (size_t)2 * p.slots * RT + blockIdx.y * 64 + 4 * f4;
  float M = kMinusBig, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  int failed = 0;
#pragma unroll 1
  for (int base = c0 + sl; base <= c1; base += kLanes * kMergeBatch) {
    float mc[kMergeBatch], lc[kMergeBatch];
    float4 oc[kMergeBatch];
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int cc = base + u * kLanes;
      mc[u] = kMinusBig;
      lc[u] = 0.f;
      oc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (cc <= c1) {
        const size_t at = (size_t)cc * RT + slot0;
        failed |= __ldcg(p.flags + cc);
        mc[u] = __ldcg(pm + at);
        lc[u] = __ldcg(pl + at);
        oc[u] = __ldcg(reinterpret_cast<const float4*>(po + at * D));
      }
    }
    float nm = M;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) nm = fmaxf(nm, mc[u]);
    const float fr = ex2(0.5f * (M - nm)), f = fr * fr;  // (L in two steps, as in the split kernel)
    L = L * fr * fr;
    O = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
    M = nm;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float er = ex2(0.5f * (mc[u] - M)), e = er * er;
      L = fmaf(lc[u] * er, er, L);
      O = make_float4(fmaf(oc[u].x, e, O.x), fmaf(oc[u].y, e, O.y), fmaf(oc[u].z, e, O.z), fmaf(oc[u].w, e, O.w));
    }
  }
  *reinterpret_cast<float4*>(&s_o[sl][4 * f4]) = O;
  if (f4 == 0) {
    s_m[sl] = M;
    s_l[sl] = L;
  }
  if (__syncthreads_or(failed)) return;  // a covering grid block gave up: o is left as it was
  if (threadIdx.x < 64) {
    float Mt = kMinusBig, Lt = 0.f, Ot = 0.f;
#pragma unroll
    for (int w = 0; w < kLanes; ++w) Mt = fmaxf(Mt, s_m[w]);
#pragma unroll
    for (int w = 0; w < kLanes; ++w) {
      const float er = ex2(0.5f * (s_m[w] - Mt)), e = er * er;
      Lt = fmaf(s_l[w] * er, er, Lt);
      Ot = fmaf(e, s_o[w][threadIdx.x], Ot);
    }
    // c1 < c0: no visible position
    p.o[((size_t)t * p.Hq + h) * D + blockIdx.y * 64 + threadIdx.x] =
        __bfloat16_as_ushort(__float2bfloat16_rn(c1 < c0 ? 0.f : Ot / Lt));
  }
}

// ================================================================= host ===

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// 3-D map of codes [pairs][L_max][D] with boxes of a unit's rows by up to 128
// bytes, swizzled by their row length; rows past L_max read as zeros.
cudaError_t codes_map(CUtensorMap* m, const void* base, int D, int L_max, int pairs) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L_max, (cuuint64_t)pairs};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)L_max * D};
  const cuuint32_t box[3] = {(cuuint32_t)(D < 128 ? D : 128), (cuuint32_t)unit_positions(D), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Groups of 8 rows per tile: as many as the average sequence's rows fill (a
// wider tile reads and converts the codes fewer times, a narrower one holds
// fewer idle rows), up to what a warp has registers for at 256 head dims, and
// up to 2 at 64, whose conversion is the smaller part. Measured, 1 / 2 / 4
// groups in us, INT8:
//   12 rows, D = 128, 64 pairs of 4096 positions   33.3 / 28.8 / 35.7
//   24 rows, D = 128, 64 pairs of 4096 positions   49.4 / 47.5 / 42.0
//   32 rows, D = 128, 4 pairs of 131,072           78.1 / 56.9 / 47.3
//   32 rows, D = 128, 4 pairs of 2048               9.7 / 10.6 / 10.7
//   24 rows, D = 64, 64 pairs of 4096              34.9 / 33.7 / 32.7
//   24 rows, D = 64, one pair of 20,000            10.2 / 11.3 / 14.3
//   32 rows, D = 256, 2 pairs of 100,000           60.1 / 50.0
int groups(int B, int T, int r, int D) {
  const long long rows = (long long)((T + B - 1) / B) * r;
  const int most = D == 128 ? 4 : 2;
  return rows <= 8 ? 1 : rows <= 16 || most == 2 ? 2 : 4;
}

// Row tiles of a call: at most one more per sequence than full tiles.
long long max_tiles(int B, int T, int r, int Hkv, int RT) {
  const long long rows = (long long)T * r, whole = rows / RT, part = rows < B ? rows : B;
  return (whole + part) * Hkv;
}

template <int D, int kNT, bool kE4m3>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const Params& prm, int grid, cudaStream_t stream) {
  static SmemLimitMemo smem_memo;
  cudaError_t e = ensure_smem(kv8_split_kernel<D, kNT, kE4m3>, Cfg<D, kNT>::kBytes, &smem_memo);
  static std::atomic<bool> known{false};
  if (e == cudaSuccess) e = launch_registers(kv8_split_kernel<D, kNT, kE4m3>, kLaunchRegs, &known);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D, kNT>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_split_kernel<D, kNT, kE4m3>, tk, tv, prm);
}

template <int D, bool kE4m3>
cudaError_t launch_groups(int nt, const CUtensorMap& tk, const CUtensorMap& tv, const Params& prm, int grid,
                          cudaStream_t stream) {
  if (nt == 1) return launch<D, 1, kE4m3>(tk, tv, prm, grid, stream);
  if (nt == 2) return launch<D, 2, kE4m3>(tk, tv, prm, grid, stream);
  if constexpr (D == 128) return launch<D, 4, kE4m3>(tk, tv, prm, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace split

size_t split_workspace_bytes(const moe_kv8_shape& s) {
  using namespace split;
  const int r = s.Hq / s.Hkv, RT = 8 * groups(s.B, s.T, r, s.D);
  const size_t slots = (size_t)kMaxCtas + max_tiles(s.B, s.T, r, s.Hkv, RT);
  return 256 + kMaxCtas * (sizeof(int32_t) + sizeof(int4)) + slots * RT * (2 + (size_t)s.D) * sizeof(float);
}

void split_steps(const moe_kv8_shape& s, long long* T) {
  const int r = s.Hq / s.Hkv;
  T[0] = (long long)(8 / r) * s.B;
  T[1] = (long long)(16 / r) * s.B;
}

moe_status launch_split(const AttnArgs& a, cudaStream_t stream) {
  using namespace split;
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice, "device query");
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  const int r = a.Hq / a.Hkv, nt = groups(a.B, a.T, r, a.D), RT = 8 * nt;
  CUtensorMap tk, tv;
  cudaError_t e = codes_map(&tk, a.k, a.D, a.L_max, a.B * a.Hkv);
  if (e == cudaSuccess) e = codes_map(&tv, a.v, a.D, a.L_max, a.B * a.Hkv);
  if (e != cudaSuccess) return cuda_fail(e, "tensor map");

  int32_t* status = static_cast<int32_t*>(a.workspace);
  int32_t* flags = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + 256);
  int4* info = reinterpret_cast<int4*>(flags + kMaxCtas);
  float* part = reinterpret_cast<float*>(info + kMaxCtas);
  const long long slots = kMaxCtas + max_tiles(a.B, a.T, r, a.Hkv, RT);
  const int shift = a.block == 16 ? 4 : a.block == 32 ? 5 : 6;
  const Params prm{a.q, a.ks, a.vs, a.offsets, a.lens, part, info, flags, slots, a.scale_log2, a.B, a.T, a.Hq, a.Hkv,
                   a.L_max, a.nblk, shift, a.q_stride, a.stalled, a.timeout_ns};
  auto go = [&](auto fp8) {
    constexpr bool kE4m3 = decltype(fp8)::value;
    return a.D == 64    ? launch_groups<64, kE4m3>(nt, tk, tv, prm, grid, stream)
           : a.D == 128 ? launch_groups<128, kE4m3>(nt, tk, tv, prm, grid, stream)
                        : launch_groups<256, kE4m3>(nt, tk, tv, prm, grid, stream);
  };
  e = a.e4m3 ? go(std::true_type{}) : go(std::false_type{});
  if (e != cudaSuccess) return cuda_fail(e, "split kernel launch");

  const MergeParams mp{a.offsets, a.lens, part, info, flags, a.o,     status, slots,
                       a.B,       a.T,    a.Hq, a.Hkv, a.D,  a.L_max, RT,     grid};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T * (unsigned)a.Hq, (unsigned)(a.D / 64));
  // An SM holds four blocks of 256 threads, or 16 of 64: more than one wave of
  // the larger would wait for the split kernel and look up the tables again.
  // Larger / smaller, both kernels in us: drafts of 16 sequences (1472 rows and
  // slices) 32.7 / 29.6; a token of 64 sequences, 2 heads of 256 (4096) 48.8 /
  // 37.1; of 8 (512) 32.6 / 35.4; one token after 32,768 positions 12.7 / 18.2.
  const bool wide = (long long)a.T * a.Hq * (a.D / 64) <= 4ll * sms;
  cfg.blockDim = dim3(wide ? 256 : 64);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg, kv8_merge_kernel<16>, mp) : cudaLaunchKernelEx(&cfg, kv8_merge_kernel<4>, mp);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "merge kernel launch");
}

}  // namespace kv8
}  // namespace bgmoe
