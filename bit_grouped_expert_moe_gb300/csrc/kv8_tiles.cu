// Attention over the 8-bit KV cache for many query tokens per sequence
// (prompts, chunks of prompts), on the 5th-generation tensor cores, sm_103a.
//
// A row is one (query token, query head of a KV head); a row tile is 256
// consecutive rows of one (sequence, KV head), 128 at 64 head dims, so the
// query heads that share keys share a tile whatever Hq / Hkv is. The positions
// that a tile's last row sees are cut into units of 128, and all units of the
// call, laid end to end in the order (sequence, KV head, row tile, position),
// are dealt out in equal contiguous runs, one per pair of blocks (per block at
// 64 head dims) of a grid with a block on every SM: a triangle of causal tiles
// and a few tiles over a long context both fill every SM. A tile that lies in
// one run is finished there; one that a run's border cuts leaves partial
// states (m, L, O) in the workspace, at most two per run, which
// kv8_tiles_merge_kernel joins in a fixed order.
//
// A pair of blocks is a cluster of two whose tensor cores work as one
// (cta_group::2): each holds 128 of the tile's rows (Q, S, P, O) and half of
// every K and V operand, so the codes are read from L2, converted and stored
// once per 256 rows: 412 us instead of 556 for the chunk below, 135 instead of
// 198 for the prompt. At 64 head dims a stage would be too small to halve.
//
// Per unit and 128 rows, 4 * 128 * 128 * D flops:
//   S = Q K^T  N = 128 positions, both operands in shared memory, S in TMEM;
//   P = 2^(x - m + 7) in fp16, written over S in TMEM;
//   O += P V   N = D (in halves of 128 at D = 256), A = P from TMEM, B = V from
//              shared memory as it lies in the cache, position by position (an
//              MN-major operand)
// S is double buffered, so the product S of the next unit runs while the softmax
// of this one is computed (TMEM: D columns of O, 2 x 128 of S).
//
// Warp roles (640 threads; setmaxnreg moves registers to the softmax):
//   warps 0-7    softmax: a thread has one row (TMEM lane) and half of the unit's
//                positions, which stay in registers from the maximum to the
//                weights; the two halves' maxima meet in shared memory. At a
//                tile's end, half of the output row each
//   warps 8-11   K codes -> fp16 operands: every thread copies its own codes into
//                shared memory stages ahead (cp.async), converts them and stores
//                them with the 128-byte swizzle
//   warps 12-15  the same for V; both bring Q in (bf16 -> fp16, a warp per row)
//   warp 16      TMEM allocation; the MMA-issuing thread (of a pair, the first
//                block's; the other block's warp tells it what is ready there)
//   warp 17      per unit, its scales and place in shared memory for the softmax
// A stage is a block's part of 128 positions x 128 head dims of K or V (16 KB of
// fp16), three of each.
//
// Bound: for 2048 queries after 16,384 positions (16 heads on 2 x 256, INT8)
// the tensor cores run 56% of a unit's 3660 cycles: a product S or O takes 1024
// and about 500 from its issue to the softmax's first read, and the softmax
// (2400) leaves the two products no more overlap. 1.39 PFLOP/s, 73% of the
// measured bf16 rate; a prompt of 4096 1.01 PFLOP/s, 53%: 56 units per pair are
// few beside the tiles' beginnings and ends. At 128 head dims the softmax
// bounds a unit: 2000 queries after 28,000 positions, 574 us, 0.83 PFLOP/s. (What
// is rare in a unit, large scores and V scales far apart, costs the softmax a
// branch: 2% of the chunk, 3% at 128 head dims, by how the code around it falls.)
//
// Codes are exact in fp16: 1024 + u (u = code + 128, by a byte permute) minus
// 1152 for int8, the conversion instruction for e4m3. Scales as in
// kv8_split.cu: with x = score + log2 s_v the weights carry V's scale and
// L = sum w / s_v (kFar: where a weight would vanish, what it stands for). The
// running maximum m of a row is raised only when a score passes it by more than
// 8 (on the base-2 scale), so that O in TMEM is rarely rescaled: w <= 2^15.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "kv8_attn.h"
#include "tiles_ptx.cuh"

namespace bgmoe {
namespace kv8 {
namespace tiles {

using namespace tc;

constexpr int kRows = 128;          // rows of a block (TMEM lanes)
constexpr int kKeys = 128;          // positions of a unit
// Of K, and of V. With 2 the chunk takes 435 us for 400; 4 of K, with smaller
// output staging in their place, 403.
constexpr int kStages = 3;
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 16, kNoteWarp = 17;
constexpr int kThreads = 20 * 32;
// Registers per thread: 96 at launch (640 x 96 in all), then 128 for the 8
// softmax warps, 88 for the 8 converting ones and 48 for the rest:
// 256 x 128 + 256 x 88 + 128 x 48 = 640 x 96. (With 120 and 96 the chunk above
// takes 417 us for 401; with 136 and 80 the prompt 171 for 148.)
constexpr int kLaunchRegs = 96, kSoftRegs = 128, kConvRegs = 88, kMmaRegs = 48;
static_assert(256 * kSoftRegs + 256 * kConvRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs, "register shares");
static_assert(kSoftRegs >= kLaunchRegs && kConvRegs <= kLaunchRegs && kMmaRegs <= kLaunchRegs,
              "the first takes what the others give");
constexpr int kGroupWarps = 4;      // converting warps of K, and of V
constexpr int kMaxCtas = 256;       // workspace bound on the grid
// A run also pays for every tile it begins (Q, the first unit's chain, the
// output), about as much as three units: the runs are cut on a scale where a
// tile with units takes kTileCost more places than units, before its first.
// A prompt of 4096 (16 heads on 2 x 256): 173, 149, 137, 140 us at 1 to 4; 16
// sequences' 8 queries over 4096 positions 53, 52, 50, 50 us.
constexpr int kTileCost = 3;
constexpr float kMinusBig = -3.402823466e38f;  // running-max start, finite: 2^(m - m_new) is never NaN
constexpr float kWeightBits = 7.f;  // weights are 2^7 at the row's m ...
constexpr float kSlack = 8.f;       // ... which scores may pass by this much
// x - m is computed in one step from the product, a x + (log2 s_v - m), so m's own
// rounding stays in it: half an fp32 step of m, which up to here is 2^-4 at most.
// Rows past it take two, the score first, rounded as m was, and the units that
// may hold such rows are told apart by a bound on their scores.
constexpr float kLargeScore = 1048576.f;  // 2^20
constexpr uint32_t kColS = 256;     // S buffers at columns 256 and 384, O from 0

// Blocks that share a tile: at 128 head dims and more a cluster of two, each
// with 128 of its 256 rows.
constexpr int tile_blocks(int D) { return D >= 128 ? 2 : 1; }

template <int D>
struct Cfg {
  static constexpr int kCtas = tile_blocks(D);
  static constexpr int kTileRows = kRows * kCtas;        // MMA M
  static constexpr int kDims = D < 128 ? D : 128;        // head dims of a stage
  static constexpr int kParts = D / kDims;               // stages of a unit's K (and V)
  static constexpr int kRaw = D == 256 ? 2 : 4;          // stages of codes on their way, of K and of V
  // A block's part of a stage: of K 128 / kCtas positions, of V kDims / kCtas
  // head dims; in slabs of 64 head dims, a 128-byte row per position.
  static constexpr int kKeyRows = kKeys / kCtas;
  static constexpr int kStageBytes = kKeyRows * kDims * 2;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kOutPitch = 80;                   // bytes: 32 bf16 and padding
  static constexpr int kOutBytes = kSoftWarps * 32 * kOutPitch;
  static constexpr int kRawBytes = kStageBytes / 2;
  static constexpr int kRawOffset = kQBytes + 2 * kStages * kStageBytes;
  static constexpr int kOutOffset = kRawOffset + 2 * kRaw * kRawBytes;
  static constexpr int kCtlOffset = kOutOffset + kOutBytes;
  static constexpr int kBytes = kCtlOffset + 4096 + 1024;  // + alignment slack
  static_assert(kStageBytes == 128 * 128 && kKeys * (kDims / kCtas) * 2 == kStageBytes, "4 pieces of a thread");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct RowConst {  // of a tile's rows, written with its Q
  uint8_t e[kRows];     // biased exponent of the row's largest magnitude
};

// What the softmax has to know of a unit, put down by a warp of its own.
struct UnitNote {
  float4 scale[8];  // of every 16 positions: s_k, log2 s_v, 1 / s_v (0 where s_v is far below others: kFar)
  int4 tile;        // lo, n, len, g of its sequence and head
  int4 place;       // first position, row tile, is the tile's last, not 0: 1 / s_v = 0, or large scores
};
constexpr int kNotes = 4;

struct Ctl {
  UnitNote note[kNotes];
  uint64_t note_full[kNotes], note_empty[kNotes];
  uint64_t full[2][kStages], empty[2][kStages];  // [K, V][stage]
  uint64_t q_full, q_empty;
  uint64_t rc_full[2], rc_empty[2];  // row constants of every second tile
  uint64_t s_full[2], p_full[2];
  // One arrival per unit, on alternate barriers. A waiter's parity is safe if
  // it cannot be two phases off: the softmax of unit u has seen S of unit u,
  // whose commit covers the products of u - 2, and those of u + 1 and u + 2
  // wait for its weights.
  uint64_t pv_done[2];
  uint64_t o_empty;       // O of a finished tile has been read
  uint64_t peer_s[2], peer_o[2];  // the other block is ready for a unit's S, for its O
  uint64_t mx_full[4];    // both halves of a lane quadrant have stored their maxima (or sums)
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
  RowConst rc[2];
  float mx[2][2][kRows];  // [unit parity][half]
};

// Where a block's run starts, for the merge kernel.
struct RunInfo {
  int tile;  // number of its first unit's tile
  int live;  // the run has units
  int b, g, rt, i;
};

struct Params {
  const uint16_t* q;
  const uint8_t* codes[2];  // K, V
  const float* ks;
  const float* vs;
  const int32_t* offsets;
  const int32_t* lens;
  uint16_t* o;
  float* part;       // two slots per run of [tile rows][D] O, then [tile rows] m and L
  RunInfo* info;     // per run
  int32_t* flags;    // [C]
  float scale_log2;
  int B, T, Hq, Hkv, L_max, nblk, shift, q_stride;
  unsigned long long rmagic;  // ceil(2^36 / r), r = Hq / Hkv
  int stalled;
  long long timeout_ns;
};

// x / r for rows x < n r of n <= 2^24 tokens and r <= 64: with the magic off by
// less than r / r from 2^36 / r, x (magic - 2^36 / r) < 2^30 < 2^36 / r keeps the
// floor, and x magic < 2^24 (2^36 + r) stays in 64 bits.
__device__ __forceinline__ int div_r(int x, unsigned long long rmagic) {
  return (int)(((unsigned long long)(unsigned)x * rmagic) >> 36);
}

constexpr size_t slot_floats(int D) { return (size_t)kRows * tile_blocks(D) * (D + 2); }

// Place in the run: unit i of the nb units of row tile rt of KV head g of
// sequence b.
struct Cursor {
  int b, g, rt, i, nb, n, len, lo;
  __device__ void sequence(const Params& p) {
    lo = ld(p.offsets + b);
    n = ld(p.offsets + b + 1) - lo;
    len = ld(p.lens + b);
  }
  __device__ bool last() const { return i == nb - 1; }
  __device__ void advance(const Params& p, int r, int RT) {
    if (++i < nb) return;
    i = 0;
    do {
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
      nb = tile_units(n, len, r, RT, kKeys, rt);
    } while (nb == 0);
  }
};

// Four codes as four fp16 values in order.
template <bool kE4m3>
__device__ __forceinline__ void convert4(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (kE4m3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p01) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p23) : "h"((uint16_t)(w >> 16)));
  } else {
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1024 + 128
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    p01 = *reinterpret_cast<const uint32_t*>(&x);
    p23 = *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) kv8_tiles_kernel(const Params p) {
  using F = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // 64-dim slabs of 128 rows x 128 bytes
  uint8_t* sR = smem + F::kQBytes;     // stages of K, then of V
  constexpr int kCtas = F::kCtas, kTileRows = F::kTileRows;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + F::kCtlOffset);
  static_assert(sizeof(Ctl) <= 4096, "control block");
  __shared__ long long s_unit[2];  // units before the run's start and end
  __shared__ Cursor s_cur;
  __shared__ int s_bad, s_tile;

  // The warp's number through a shuffle, which the compiler knows to be
  // uniform: the roles' loops then run on uniform registers, where the MMA
  // instructions take their descriptors from.
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int C = gridDim.x / kCtas, c = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;  // runs, run, block of its tiles
  const int r = p.Hq / p.Hkv;

  if (threadIdx.x == 32) {
    mbar_init(&ctl->q_full, 2 * kGroupWarps);
    for (int i = 0; i < kNotes; ++i) {
      mbar_init(&ctl->note_full[i], 1);
      mbar_init(&ctl->note_empty[i], kSoftWarps);
    }
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&ctl->full[i][s], kGroupWarps);
        mbar_init(&ctl->empty[i][s], 1);
      }
      mbar_init(&ctl->rc_full[i], 2 * kGroupWarps);
      mbar_init(&ctl->rc_empty[i], kSoftWarps);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], kSoftWarps);
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->peer_s[i], 1);
      mbar_init(&ctl->peer_o[i], 1);
    }
    mbar_init(&ctl->o_empty, kSoftWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&ctl->mx_full[i], 2);
    mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  // Launched with programmatic dependent launch: wait for the kernels before
  // this one, then let this call's merge launch (it waits in turn).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 1 || warp == 2) {  // the run's start and its end
    Place k;
    const bool ok = find_run(p.offsets, p.lens, p.B, p.T, p.Hkv, p.L_max, r, kTileRows, kKeys, kTileCost, c + warp - 1,
                             C, &k);
    if (lane == 0) {
      s_unit[warp - 1] = k.units;
      if (warp == 1) {
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
        }
        s_cur = cur;
        s_tile = k.tile;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool live = !s_bad && s_unit[0] < s_unit[1];
    if (rank == 0) p.info[c] = RunInfo{s_tile, live, s_cur.b, s_cur.g, s_cur.rt, s_cur.i};
    if (!live) p.flags[blockIdx.x] = s_bad ? (int32_t)MOE_ERR_INVALID_ARG : 0;
  }
  if (s_bad) return;
  // Queries that see nothing (more queries than positions): o = 0.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int lo = ld(p.offsets + b), hi = ld(p.offsets + b + 1), len = ld(p.lens + b);
    const size_t pieces = (size_t)max(0, hi - lo - len) * p.Hq * (D / 8);
    uint4* z = reinterpret_cast<uint4*>(p.o + (size_t)lo * p.Hq * D);
    for (size_t i = threadIdx.x; i < pieces; i += kThreads) z[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (s_unit[0] >= s_unit[1]) return;  // both blocks of a run alike
  if (warp == kMmaWarp) alloc_columns<kCtas>(&ctl->tmem);
  tc_fence_before();
  tile_barrier<kCtas>();  // the barriers and the columns of both blocks are there
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
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

  if (warp >= kMmaWarp) {
    fewer_registers<kMmaRegs>();
    if (warp == kMmaWarp) {
      // ----------------------------------------------------- MMA issuer
      // With two blocks the leader's warp issues for both; the other's goes
      // through the same steps, waits for what its own block has to have ready
      // and passes that on as one arrival. (With the block's warps arriving on
      // the leader's barriers themselves, each by a release at cluster scope
      // that waited for its loads first, the chunk took 549 us; through this
      // warp 470; with the restricted release of arrive_leader 436.)
      constexpr uint32_t idesc_s = idesc_f16_f32(kTileRows, kKeys);
      constexpr uint32_t idesc_o = idesc_f16_f32(kTileRows, F::kDims) | (1u << 16);  // B is MN-major
      const uint64_t dq = sw128_desc(smem_u32(sQ));
      const uint32_t leader = elect_one();
      const uint64_t dk = sw128_desc(smem_u32(sR));
      const uint64_t dv = sw128_mn_desc(smem_u32(sR) + kStages * F::kStageBytes, kKeys * 128);
      int tq = 0, to = 0;              // tiles whose Q has been waited for, whose O has been started
      Cursor nxt = cur;
      // stage h of unit u, and its phase
      auto stage = [](int u, int h) { return (u * F::kParts + h) % kStages; };
      auto phase = [](int u, int h) { return (uint32_t)((u * F::kParts + h) / kStages) & 1u; };
      // Waits until a step of unit u may begin: its stages of K or V, the
      // softmax's or Q's barrier `own` (if any), the other block's arrival;
      // all tested together. The other block's warp passes its readiness on.
      // (An arrival for unit u + 2 comes after the leader's step of unit u: two
      // barriers in turn will do.)
      auto ready = [&](int kv, int u, uint64_t* own, uint32_t parity, uint64_t* peer) -> bool {
        bool all = own == nullptr || mbar_test_wait(own, parity);
#pragma unroll
        for (int h = 0; h < F::kParts; ++h) all = mbar_test_wait(&ctl->full[kv][stage(u, h)], phase(u, h)) && all;
        const bool listens = kCtas == 2 && rank == 0;
        if (listens) all = test_cluster(peer, (u >> 1) & 1) && all;
        if (!__all_sync(0xffffffffu, all)) {
          if (own != nullptr && !warp_wait(own, parity)) return false;
          for (int h = 0; h < F::kParts; ++h)
            if (!warp_wait(&ctl->full[kv][stage(u, h)], phase(u, h))) return false;
          if (listens && !warp_wait(peer, (u >> 1) & 1)) return false;
          // (a test at cluster scope, for the fence below to follow on)
          if (listens && !__all_sync(0xffffffffu, test_cluster(peer, (u >> 1) & 1))) return false;
        }
        tc_fence_after();
        if (listens) acquire_peer();
        if (kCtas == 2 && rank != 0) {
          tc_fence_before();
          if (lane == 0) arrive_leader(peer);
        }
        return true;
      };
      auto score = [&](int u, bool first, bool ends) -> bool {  // S of unit u
        if (!ready(0, u, first ? &ctl->q_full : nullptr, tq & 1, &ctl->peer_s[u & 1])) return false;
        tq += first;
        if (rank != 0) return true;
        const uint32_t d = tmem + kColS + 128 * (u & 1);
#pragma unroll
        for (int h = 0; h < F::kParts; ++h) {
          const int st = stage(u, h);
#pragma unroll
          for (int kk = 0; kk < F::kDims / 16; ++kk) {
            const uint32_t slab = kk >> 2, in = (kk & 3) * 2;  // 64-dim slabs
            mma_ss<kCtas>(d, dq + (h * (F::kDims / 64) + slab) * (kRows * 128 / 16) + in,
                          dk + st * (F::kStageBytes / 16) + slab * (F::kKeyRows * 128 / 16) + in, idesc_s,
                          kk > 0 || h > 0, leader);
          }
          commit<kCtas>(&ctl->empty[0][st], leader);
        }
        commit<kCtas>(&ctl->s_full[u & 1], leader);
        if (ends) commit<kCtas>(&ctl->q_empty, leader);
        return true;
      };
      auto output = [&](int u, bool first) -> bool {  // O of unit u
        if (first && to++ > 0 && !warp_wait(&ctl->o_empty, (to - 2) & 1)) return false;
        if (!ready(1, u, &ctl->p_full[u & 1], (u >> 1) & 1, &ctl->peer_o[u & 1])) return false;
        if (rank != 0) return true;
        const uint32_t a = tmem + kColS + 128 * (u & 1);
#pragma unroll
        for (int h = 0; h < F::kParts; ++h) {
          const int st = stage(u, h);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts<kCtas>(tmem + h * F::kDims, a + kk * 8, dv + st * (F::kStageBytes / 16) + kk * (16 * 128 / 16),
                          idesc_o, kk > 0 ? 1u : (uint32_t)!first, leader);
          commit<kCtas>(&ctl->empty[1][st], leader);
        }
        commit<kCtas>(&ctl->pv_done[u & 1], leader);
        return true;
      };
      // S of unit u + 1 goes ahead of O of unit u, whose weights the softmax
      // makes meanwhile; not where u + 1 starts a tile, whose Q may be long in
      // coming. (One call site each: the code stays short.)
      bool ok = true, sfirst = true, ofirst = true;  // unit su, ou starts a tile (in this run)
      int su = 0, ou = 0;              // units scored and put out so far
#pragma unroll 1
      while (ok && ou < U) {
        if (su < U && su <= ou + 1 && (su == ou || !sfirst)) {
          const bool last = nxt.last();
          ok = score(su, sfirst, last || su + 1 == U);
          sfirst = last;
          if (++su < U) nxt.advance(p, r, F::kTileRows);
        } else {
          ok = output(ou, ofirst);
          // with su == ou + 1 the next unit's sfirst is this one's end; with
          // su == ou + 2 unit ou + 1 is of the same tile
          ++ou;
          ofirst = su == ou && sfirst;
        }
      }
      if (rank == 0) commit<kCtas>(&ctl->mma_done, leader);
    } else if (warp == kNoteWarp) {
      // ----------------------------------------------------- unit notes
      Cursor k = cur;
      uint32_t top = 0u;  // the tile's largest V scale so far (positive floats compare as their bits)
      float most = 0.f;   // its scores' bound, but for the K scale: 2 is q's largest magnitude, 448 the codes'
      int tile = 0;
      bool begins = true;
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int s = u % kNotes;
        const int pos = min(k.i * kKeys + 16 * (lane & 7), k.len - 1);
        const size_t at = (size_t)(k.b * p.Hkv + k.g) * p.nblk + (pos >> p.shift);
        const float sk = ld(p.ks + at), v = ld(p.vs + at), sv = v > 0.f ? v : kScaleFloor;
        top = max(top, __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(v, 0.f))));
        const int far = __ballot_sync(0xffffffffu, sv < kFar * __uint_as_float(top)) & 0xFF;
        if (begins) {  // the rows' exponents come with Q; the softmax reads them after this note
          if (!warp_wait(&ctl->rc_full[tile & 1], (tile >> 1) & 1)) break;
          const uint32_t e = reinterpret_cast<const uint32_t*>(ctl->rc[tile & 1].e)[lane];  // of four rows
          const uint32_t e2 = __vmaxu4(e, e >> 16), e1 = __vmaxu4(e2, e2 >> 8) & 0xFF;
          most = p.scale_log2 * (2.f * 448.f * D) * __uint_as_float(max(__reduce_max_sync(0xffffffffu, e1), 1u) << 23);
          ++tile;
        }
        begins = k.last();
        const int large = __any_sync(0xffffffffu, !(most * sk < kLargeScore)) ? 0x100 : 0;
        if (u >= kNotes && !warp_wait(&ctl->note_empty[s], (u / kNotes - 1) & 1)) break;
        const float rsv = far >> lane & 1 ? 0.f : __fdividef(1.f, sv);
        if (lane < 8) ctl->note[s].scale[lane] = make_float4(sk, __log2f(sv), rsv, 0.f);
        if (lane == 8) ctl->note[s].tile = make_int4(k.lo, k.n, k.len, k.g);
        if (lane == 9) ctl->note[s].place = make_int4(k.i * kKeys, k.rt, k.last(), far | large);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->note_full[s]);
        if (begins) top = 0u;
        if (u + 1 < U) k.advance(p, r, F::kTileRows);
      }
    }
  } else if (warp < kSoftWarps) {
    // --------------------------------------------------------- softmax
    more_registers<kSoftRegs>();
    const int quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    float m = kMinusBig, l = 0.f, rs = 0.f;
    int see = 0, tile = 0, met = 0;
    bool fresh = true, mid = cur.i > 0;  // the tile's first unit in this run; the tile began in an earlier run
    // this thread's value and its partner's, once both are there
    auto meet = [&](float v, float& other) -> bool {
      ctl->mx[met & 1][half][row] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->mx_full[quad]);
      if (!warp_wait(&ctl->mx_full[quad], met & 1)) return false;
      other = ctl->mx[met & 1][half ^ 1][row];
      ++met;
      return true;
    };
    int4 seq = make_int4(0, 0, 0, 0);  // lo, n, len, g of the tile
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      const int ns = u % kNotes;
      if (!warp_wait(&ctl->note_full[ns], (u / kNotes) & 1)) break;
      const int4 place = ctl->note[ns].place;
      float4 sc[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) sc[h] = ctl->note[ns].scale[4 * half + h];
      if (fresh) {
        seq = ctl->note[ns].tile;
        if (!warp_wait(&ctl->rc_full[tile & 1], (tile >> 1) & 1)) break;
        const RowConst& rc = ctl->rc[tile & 1];
        const int e = rc.e[row], rho = place.y * kTileRows + rank * kRows + row;
        __syncwarp();
        rs = p.scale_log2 * __uint_as_float(e > 0 ? (uint32_t)e << 23 : 0x00400000u);  // 2^(e - 127)
        see = rho < seq.y * r ? max(seq.z - seq.y + div_r(rho, p.rmagic) + 1, 0) : 0;
        if (lane == 0) mbar_arrive(&ctl->rc_empty[tile & 1]);
        m = kMinusBig;
        l = 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->note_empty[ns]);
      if (!warp_wait(&ctl->s_full[u & 1], (u >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t ts = lane_addr + kColS + 128 * (u & 1);
      uint32_t x[64];
      tmem_ld_64(ts + 64 * half, x);
      // Scores on the base-2 scale, with V's scale: a x + b, a and b per 16
      // positions. a is kept above zero, so hidden positions (x = -inf) stay
      // hidden and a group's largest x gives its largest score.
      const int left = see - place.x - 64 * half;  // visible positions from this half's first on
      if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= left) x[e] = 0xFF800000u;  // -inf
      }
      float mx = -INFINITY;
      float a[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        a[h] = fmaxf(rs * sc[h].x, 1e-35f);
        float g = fmaxf(__uint_as_float(x[16 * h]), __uint_as_float(x[16 * h + 1]));
#pragma unroll
        for (int e = 16 * h + 2; e < 16 * h + 16; e += 2)
          g = fmaxf(g, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
        mx = fmaxf(mx, fmaf(g, a[h], sc[h].y));
      }
      float other;
      if (!meet(mx, other)) break;
      mx = fmaxf(mx, other);
      if (fresh) {
        m = fmaxf(mx, kMinusBig);
      } else if (__any_sync(0xffffffffu, mx > m + kSlack)) {
        // O and L to the new maximum, once the products of the last unit are in
        const float nm = mx > m + kSlack ? mx : m, root = ex2(0.5f * (m - nm)), f = root * root;
        m = nm;
        l = l * root * root;
        if (!warp_wait(&ctl->pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = half * (D / 2); j < (half + 1) * (D / 2); j += 16) {
          uint32_t w[16];
          tmem_ld_16(lane_addr + j, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
          tmem_st_16(lane_addr + j, w);
        }
      }
      // weights, over S (both halves have read it)
      const float top = kWeightBits - m;
      if (place.w) {  // the whole warp alike
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (sc[h].z == 0.f) {
            const float lift = kLiftBits - sc[h].y;
            float s = 0.f;
#pragma unroll
            for (int e = 16 * h; e < 16 * h + 16; ++e)
              s += ex2(fmaf(__uint_as_float(x[e]), a[h], sc[h].y) + top + lift);
            l = fmaf(s, kUnlift, l);
          }
        // Rows of large scores: a x + b with a = 1, b = 0 from here on, or NaN where m
        // is infinite. (A score that m + kSlack, rounded, let pass stays within fp16.)
        if (fabsf(m) > kLargeScore && m > kMinusBig) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int e = 16 * h; e < 16 * h + 16; ++e)
              x[e] = __float_as_uint(
                  fminf(fmaf(__uint_as_float(x[e]), a[h], sc[h].y) + top, kWeightBits + kSlack));
            a[h] = 1.f;
            sc[h].y = -top;
          }
        }
      }
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint64_t s2 = 0ull;
        const float bt = sc[h].y + top;
        const uint64_t a2 = pack2(a[h], a[h]), b2 = pack2(bt, bt);
#pragma unroll
        for (int e = 16 * h; e < 16 * h + 16; e += 2) {
          const float2 y = unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), a2, b2));
          const float w0 = ex2(y.x), w1 = ex2(y.y);
          s2 = add2(s2, pack2(w0, w1));
          w[e / 2] = pack_f16(w0, w1);
        }
        const float2 s = unpack2(s2);
        l = fmaf(s.x + s.y, sc[h].z, l);
      }
      tmem_st_32(ts + 32 * half, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[u & 1]);

      const bool ends = place.z != 0;
      fresh = ends;
      if (ends || u + 1 == U) {
        // ---- the run leaves this tile: its rows' outputs, or the partial state
        if (!meet(l, other)) break;
        l += other;
        if (!warp_wait(&ctl->pv_done[u & 1], (u >> 1) & 1)) break;
        tc_fence_after();
        const int d0 = half * (D / 2);
        if (!mid && ends) {
          const float inv = see > 0 ? 1.f / l : 0.f;
          // 32 rows by 32 dims at a time through shared memory: 4 lanes write
          // a row's 64 bytes, 8 rows at once
          const uint32_t stage = smem_u32(smem + F::kOutOffset) + warp * (32 * F::kOutPitch);
          uint16_t* orow[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rk = place.y * kTileRows + rank * kRows + quad * 32 + 8 * k + (lane >> 2);
            const int tok = div_r(rk, p.rmagic);
            const bool live = rk < seq.y * r && seq.z - seq.y + tok >= 0;
            uint16_t* at = p.o + ((size_t)(seq.x + tok) * p.Hq + (size_t)seq.w * r + rk - tok * r) * D + 8 * (lane & 3);
            orow[k] = live ? at : nullptr;
          }
#pragma unroll 1
          for (int j = d0; j < d0 + D / 2; j += 32) {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              uint32_t v[16];
              tmem_ld_16(lane_addr + j + h, v);
#pragma unroll
              for (int e = 0; e < 16; e += 8) {
                uint32_t z[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(v[e + 2 * k]) * inv,
                                                                 __uint_as_float(v[e + 2 * k + 1]) * inv);
                  z[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                sts128(stage + lane * F::kOutPitch + 2 * (h + e), z[0], z[1], z[2], z[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 y = lds128(stage + (8 * k + (lane >> 2)) * F::kOutPitch + 16 * (lane & 3));
              if (orow[k]) *reinterpret_cast<uint4*>(orow[k] + j) = y;
            }
          }
        } else {
          // 32 rows by 16 dims at a time, the same way
          float* part = p.part + (size_t)(2 * c + (mid ? 0 : 1)) * slot_floats(D);
          const uint32_t stage = smem_u32(smem + F::kOutOffset) + warp * (32 * F::kOutPitch);
          float* prow = part + (size_t)(rank * kRows + quad * 32 + (lane >> 2)) * D + 4 * (lane & 3);
#pragma unroll 1
          for (int j = d0; j < d0 + D / 2; j += 16) {
            uint32_t v[16];
            tmem_ld_16(lane_addr + j, v);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              sts128(stage + lane * F::kOutPitch + 4 * e, v[e], v[e + 1], v[e + 2], v[e + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(prow + (size_t)(8 * k) * D + j) =
                  lds128(stage + (8 * k + (lane >> 2)) * F::kOutPitch + 16 * (lane & 3));
          }
          if (half == 0) {
            part[(size_t)D * kTileRows + rank * kRows + row] = m;
            part[(size_t)(D + 1) * kTileRows + rank * kRows + row] = l;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_empty);
        ++tile;
        mid = false;
        fresh = true;
      }
    }
  } else {
    // ---------------------------------------------- codes -> fp16 operands
    fewer_registers<kConvRegs>();
    const int kv = (warp - kSoftWarps) / kGroupWarps;            // 0: K (and Q), 1: V
    const int t = threadIdx.x - 32 * (kSoftWarps + kv * kGroupWarps);
    // This thread's four pieces of a stage, 16 head dims of a position each, 4096
    // bytes apart in the stage: of V (and at D = 64) positions key, key + 32, +
    // 64, + 96 of the block's 64 head dims; of K positions key and key + 32 of
    // the block's 64, then the same of the next 64 head dims. 8 lanes that
    // store together have two neighbouring positions, which the swizzle keeps
    // on different banks.
    const int piece = t & 3, key = t >> 2;
    const bool by_dims = kCtas == 2 && kv == 0;
    const uint32_t stage0 = smem_u32(sR) + kv * (kStages * F::kStageBytes) + key * 128;
    const uint32_t ch = (uint32_t)piece * 2, sw = key & 7;
    const uint32_t b0 = stage0 + ((ch ^ sw) << 4), b1 = stage0 + (((ch + 1) ^ sw) << 4);
    const int key0 = by_dims ? rank * F::kKeyRows : 0;                // the block's first position and head dim
    const int dim0 = kCtas == 2 && kv == 1 ? rank * (F::kDims / kCtas) : 0;
    const int second = by_dims ? 64 : 64 * D;                         // from the first two pieces to the others

    // A thread's codes come through shared memory of its own (cp.async), kRaw
    // stages ahead: loads into registers are waited for together with those
    // issued after them. Positions past the context are code 0 of the format
    // or, as INT8, -128: finite and not seen either way.
    const uint32_t raw = smem_u32(smem + F::kRawOffset) + kv * (F::kRaw * F::kRawBytes) + t * 16;
    Cursor cn = cur;             // unit of the next load
    int hn = 0, left = U * F::kParts;  // its stage; stages to load
    const uint8_t* src;          // this thread's first piece of the unit
    int keys, keys2;             // positions from its first piece, and from its third, on
    auto limits = [&]() {
      keys = cn.len - cn.i * kKeys - key0 - key;
      keys2 = by_dims ? keys : keys - 64;
    };
    auto place = [&]() {
      src = p.codes[kv] + ((size_t)(cn.b * p.Hkv + cn.g) * p.L_max + (size_t)cn.i * kKeys + key0 + key) * D + dim0 +
            piece * 16;
      limits();
    };
    place();
    auto load_stage = [&](int j) {
      if (left > 0) {
        const uint32_t to = raw + (j % F::kRaw) * F::kRawBytes;
        const uint8_t* from = src + hn * F::kDims;
        load16(to, from, keys > 0);
        load16(to + 2048, from + 32 * D, keys > 32);
        load16(to + 4096, from + second, keys2 > 0);
        load16(to + 6144, from + second + 32 * D, keys2 > 32);
        --left;
        if (++hn == F::kParts && left > 0) {
          hn = 0;
          if (cn.last()) {
            cn.advance(p, r, F::kTileRows);
            place();
          } else {
            ++cn.i;
            src += kKeys * D;
            limits();
          }
        }
      }
      cp_async_commit();  // an empty group at the end: the count of groups stays
    };
#pragma unroll 1
    for (int j = 0; j < F::kRaw; ++j) load_stage(j);

    // Q of the tile at a cursor: D / 8 lanes per row, 16 bytes each
    int tile = 0;
    constexpr int kLanes = D / 8, kAtOnce = 256 / D, kBatch = 4;    // lanes per row; rows of a load; loads in flight
    constexpr int kQRows = kRows / (2 * kGroupWarps * kAtOnce);     // loads of a lane
    const int ln = lane % kLanes, qrow = (warp - kSoftWarps) * (kRows / (2 * kGroupWarps)) + lane / kLanes;
    auto load_rows = [&](const Cursor& k, int base, uint4 (&v)[kBatch]) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int rho = k.rt * kTileRows + rank * kRows + qrow + (base + i) * kAtOnce, tok = div_r(rho, p.rmagic);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        ldg128_if<0>(v[i], reinterpret_cast<const uint8_t*>(p.q + (size_t)(k.lo + tok) * p.q_stride +
                                                            (size_t)(k.g * r + rho - tok * r) * D + ln * 8),
                     rho < k.n * r);
      }
    };
    auto load_q = [&](const Cursor& k) -> bool {
      uint4 v[kBatch];
      load_rows(k, 0, v);  // on their way while the last tile's products end
      if (tile > 0 && !warp_wait(&ctl->q_empty, (tile - 1) & 1)) return false;
      if (tile > 1 && !warp_wait(&ctl->rc_empty[tile & 1], ((tile >> 1) - 1) & 1)) return false;
      tc_fence_after();
      RowConst& rc = ctl->rc[tile & 1];
#pragma unroll 2  // with all at once, a value of the stages' loop is spilled (the chunk above 412 us for 399)
      for (int base = 0; base < kQRows; base += kBatch) {
        if (base > 0) load_rows(k, base, v);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = qrow + (base + i) * kAtOnce;
          uint32_t mx = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
          mx = max(mx & 0xFFFFu, mx >> 16);
          if (kLanes == 32) {
            mx = __reduce_max_sync(0xffffffffu, mx);
          } else {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          }
          const int e = min((int)(mx >> 7), 253);
          const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^-(e - 127)
          const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = pack_f16(__uint_as_float(in[j] << 16) * down, __uint_as_float(in[j] & 0xFFFF0000u) * down);
          sts128(smem_u32(sQ) + (ln >> 3) * (kRows * 128) + row * 128 + (((ln & 7) ^ (row & 7)) << 4), x[0], x[1], x[2],
                 x[3]);
          if (ln == 0) rc.e[row] = (uint8_t)e;
        }
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

    bool ok = kv == 0 || (int)blockIdx.x != p.stalled, fresh = true;
    Cursor k = cur;
    int st = 0;
    uint32_t free = 1;           // parity of a stage's last use (a first use waits for nothing)
#pragma unroll 1
    for (int u = 0; ok && u < U; ++u) {
      if (fresh && !load_q(k)) break;
      fresh = k.last();
      if (u + 1 < U) k.advance(p, r, F::kTileRows);
#pragma unroll 1
      for (int h = 0; h < F::kParts; ++h) {
        const int j = u * F::kParts + h;
        cp_async_wait<F::kRaw - 1>();
        const uint32_t from = raw + (j % F::kRaw) * F::kRawBytes;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = lds128(from + 2048 * i);
        ok = warp_wait(&ctl->empty[kv][st], free);
        if (!ok) break;
        tc_fence_after();
        const uint32_t to = st * F::kStageBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[8];
          convert4<kE4m3>(w[i].x, x[0], x[1]);
          convert4<kE4m3>(w[i].y, x[2], x[3]);
          convert4<kE4m3>(w[i].z, x[4], x[5]);
          convert4<kE4m3>(w[i].w, x[6], x[7]);
          sts128(b0 + to + 4096 * i, x[0], x[1], x[2], x[3]);
          sts128(b1 + to + 4096 * i, x[4], x[5], x[6], x[7]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[kv][st]);
        load_stage(j);           // into the slot just read
        if (++st == kStages) {
          st = 0;
          free ^= 1;
        }
      }
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    int dummy = 0;  // no MMA may still be running when TMEM is freed
    mbar_wait(&ctl->mma_done, 0, &dummy, global_timer_ns() + 2 * (uint64_t)p.timeout_ns);
    tc_fence_after();
  }
  tile_barrier<kCtas>();  // nor a block's shared memory and barriers be gone while the other uses them
  if (warp == kMmaWarp) free_columns<kCtas>(tmem);
  if (threadIdx.x == 0) p.flags[blockIdx.x] = *abort_flag ? (int32_t)MOE_ERR_DEVICE_TIMEOUT : 0;
}

struct MergeParams {
  const int32_t* offsets;
  const int32_t* lens;
  const float* part;
  const RunInfo* info;
  const int32_t* flags;
  uint16_t* o;
  int32_t* status;
  int Hq, Hkv, D, C, ctas;  // C: runs
};

// Rows of a block, a warp each. 4, 8, 16, 32: a prompt of 4096 takes 133.1,
// 132.8, 133.0, 140.9 us, 16 sequences' 8 queries 48.2, 47.4, 48.4, 48.2.
constexpr int kMergeRows = 8;
constexpr int kMergeThreads = 32 * kMergeRows;

// Block (c, y): if run c is the second of the runs that share a tile, the
// tile's rows 8 y .. + 7. The first run of a tile left its state in its second
// slot (a tile that the run's end cuts), the others in their first.
__global__ void __launch_bounds__(kMergeThreads) kv8_tiles_merge_kernel(const MergeParams p) {
  __shared__ int s_first, s_c0, s_later;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, C = p.C, t = threadIdx.x, lane = t & 31;
  if (c == 0 && blockIdx.y == 0) {
    // the call's status: the outcome of the lowest-numbered grid block that failed
    const int blocks = C * p.ctas;
    if (t == 0) s_first = blocks;
    __syncthreads();
    for (int cc = t; cc < blocks; cc += kMergeThreads)
      if (__ldcg(p.flags + cc) != 0) atomicMin(&s_first, cc);
    __syncthreads();
    if (t == 0) *p.status = s_first == blocks ? 0 : __ldcg(p.flags + s_first);
  }
  // Run c is the tile's second if it starts inside the tile and the last live
  // run before it does not, or does at the first unit; the runs after it that
  // start in the tile follow one another.
  const RunInfo f = p.info[c];
  if (!f.live || f.i == 0) return;
  if (t == 0) s_c0 = -1;
  __syncthreads();
  int later = 0;
  for (int cc = t; cc < C; cc += kMergeThreads) {
    const int2 x = __ldcg(reinterpret_cast<const int2*>(&p.info[cc]));  // tile, live
    if (!x.y) continue;
    if (cc < c) atomicMax(&s_c0, cc);
    else if (x.x == f.tile) ++later;
  }
  if (t == 0) s_later = 0;
  __syncthreads();
  if (later) atomicAdd(&s_later, later);
  __syncthreads();
  const int c0 = s_c0, c1 = c + s_later - 1;
  if (c0 < 0) return;
  const RunInfo f0 = p.info[c0];
  if (f0.tile == f.tile && f0.i > 0) return;  // a later one of the tile's runs
  const int r = p.Hq / p.Hkv, D = p.D, row = blockIdx.y * kMergeRows + (t >> 5);
  const int lo = ld(p.offsets + f.b), n = ld(p.offsets + f.b + 1) - lo, len = ld(p.lens + f.b);
  const int rows = kRows * p.ctas, rho = f.rt * rows + row, tok = rho / r;
  if (rho >= n * r || len - n + tok < 0) return;
  auto slot = [&](int cc) { return p.part + (size_t)(2 * cc + (cc == c0 ? 1 : 0)) * slot_floats(D); };
  // lane k weighs the states of runs c0 + k, c0 + 32 + k, ...
  float M = kMinusBig;
  bool failed = false;
  for (int cc = c0 + lane; cc <= c1; cc += 32) {
    for (int k = 0; k < p.ctas; ++k) failed |= __ldcg(p.flags + cc * p.ctas + k) != 0;
    M = fmaxf(M, __ldcg(slot(cc) + (size_t)D * rows + row));
  }
  if (__any_sync(0xffffffffu, failed)) return;  // a run gave up: o is left as it was
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, acc[8];  // head dims lane * D / 32 .. of the row
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  const int per = D / 32;
  for (int base = c0; base <= c1; base += 32) {
    const int mine = base + lane;
    const float root = mine <= c1 ? exp2f(0.5f * (__ldcg(slot(mine) + (size_t)D * rows + row) - M)) : 0.f;
    const float e = root * root;
    float l = mine <= c1 ? __ldcg(slot(mine) + (size_t)(D + 1) * rows + row) * root * root : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    L += l;
    for (int cc = base; cc <= min(c1, base + 31); ++cc) {
      const float w = __shfl_sync(0xffffffffu, e, cc - base);
      const float* o = slot(cc) + (size_t)row * D + lane * per;
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        if (i < per) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(o + i));
          acc[i] = fmaf(w, x.x, acc[i]);
          acc[i + 1] = fmaf(w, x.y, acc[i + 1]);
        }
    }
  }
  const float inv = 1.f / L;
  uint16_t* out = p.o + ((size_t)(lo + tok) * p.Hq + (size_t)f.g * r + rho - tok * r) * D + lane * per;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    if (i < per) *reinterpret_cast<__nv_bfloat162*>(out + i) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
}

}  // namespace tiles

size_t tiles_workspace_bytes(const moe_kv8_shape& s) {
  using namespace tiles;
  return 256 + kMaxCtas * (sizeof(int32_t) + sizeof(RunInfo)) +
         2 * (kMaxCtas / tile_blocks(s.D)) * slot_floats(s.D) * sizeof(float);
}

moe_status launch_tiles(const AttnArgs& a, cudaStream_t stream) {
  using namespace tiles;
  const int sms = sm_count();
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice, "device query");
  const int ctas = tile_blocks(a.D), runs = (sms < kMaxCtas ? sms : kMaxCtas) / ctas;
  if (runs < 1) return cuda_fail(cudaErrorInvalidDevice, "multiprocessors");
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  int32_t* flags = reinterpret_cast<int32_t*>(ws + 256);
  RunInfo* info = reinterpret_cast<RunInfo*>(ws + 256 + kMaxCtas * sizeof(int32_t));
  float* part = reinterpret_cast<float*>(ws + 256 + kMaxCtas * (sizeof(int32_t) + sizeof(RunInfo)));
  const int shift = a.block == 16 ? 4 : a.block == 32 ? 5 : 6;
  const Params prm{a.q, {a.k, a.v}, a.ks, a.vs, a.offsets, a.lens, a.o, part, info, flags, a.scale_log2,
                   a.B, a.T, a.Hq, a.Hkv, a.L_max, a.nblk, shift, a.q_stride,
                   ((1ull << 36) + a.Hq / a.Hkv - 1) / (a.Hq / a.Hkv), a.stalled, a.timeout_ns};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(runs * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto go = [&](auto d, auto fp8) -> cudaError_t {
    constexpr int D = decltype(d)::value;
    constexpr bool kE4m3 = decltype(fp8)::value;
    static SmemLimitMemo smem_memo;
    static std::atomic<bool> known{false};
    cudaError_t e = ensure_smem(kv8_tiles_kernel<D, kE4m3>, Cfg<D>::kBytes, &smem_memo);
    if (e == cudaSuccess) e = launch_registers(kv8_tiles_kernel<D, kE4m3>, kLaunchRegs, &known);
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
  const MergeParams mp{a.offsets, a.lens, part, info, flags, a.o, status, a.Hq, a.Hkv, a.D, runs, ctas};
  cfg.gridDim = dim3((unsigned)runs, (unsigned)(kRows * ctas / kMergeRows));
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, kv8_tiles_merge_kernel, mp);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "merge kernel launch");
}

}  // namespace kv8
}  // namespace bgmoe
