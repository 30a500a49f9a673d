// Attention over the paged bf16 cache (include/paged.h): causal, or for trees
// of drafts, from one query token per sequence to whole prompts, on the
// 5th-generation tensor cores, sm_103a.
//
// A row is one (query token, query head of a KV head); a row tile is 128
// consecutive rows of one (sequence, KV head), or 256 on a pair of blocks. The
// positions that a tile's last row sees are cut into units of 128, and all
// units of the call, laid end to end in the order (sequence, KV head, row tile,
// position), are dealt out in equal contiguous runs, one per block (per pair)
// of a grid with a block on every SM (kv8_attn.h has the arithmetic). A tile that
// lies in one run is finished there; one that a run's border cuts leaves partial
// states (m, L, O) in the workspace, at most two per run, which
// paged_merge_kernel joins in a fixed order.
//
// Per unit and 128 rows, 4 * 128 * 128 * D flops:
//   S = Q K^T  N = 128 positions, both operands in shared memory, S in TMEM;
//   P = 2^(scale log2(e) (S - m)) in bf16, written over S in TMEM;
//   O += P V   N = D, A = P from TMEM, B = V from shared memory as it lies in
//              its page, position by position (an MN-major operand)
// The products S of the next units run while the softmax of one is computed: TMEM
// has D columns of O and two buffers of S, at 64 and 128 head dims three. (A
// softmax needs 2000 cycles from S to P, and with two S of the next unit but one
// waits in line behind O of this: 2000 tokens after 28,000 positions at 128 take
// 376 us for 364.) At 64 head dims the two halves of a unit's positions have an
// O each, and a maximum and a sum, which meet at a tile's end only: the halves
// of the softmax need not wait for one another (327 -> 316 us; at 128 there
// is room for it with two buffers of S, 372 us for 363).
//
// One row or 128: a product costs the same, and its 2 x 1024 cycles of a unit at
// D = 256 are less than half of what its 128 KB take to come from HBM. So a
// single token of a sequence runs here, too, with the rows that are not there
// left out of the softmax and of the partial states.
//
// Warp roles (512 threads):
//   warps 0-7    softmax: a thread has one row (TMEM lane) and half of the unit's
//                positions, which stay in registers from the maximum to the
//                weights; the two halves' maxima meet in shared memory. At a
//                tile's end, half of the output row each. (Whole rows of every
//                other unit, half of them read twice, are no quicker: 366 us for 356)
//   warps 8-11   Q into shared memory; values of V that no row, or not every row,
//                sees and that are no finite numbers out of it (0 * NaN is NaN)
//   warp 12      TMEM allocation; the MMA-issuing thread (of a pair, the first
//                block's; the other block's warp tells it what is ready there)
//   warps 13, 14 K and V by TMA, a stage each in turn (page numbers from the table
//                32 at a time, positions past the context as zeros). One warp has
//                some 130 cycles a box: 2000 tokens after 28,000 positions in
//                pages of 16, 32, 64 (16 heads on 4 of 128) 509, 425, 354 us for
//                385, 356, 355
// The ring's stages (16 KB) hold K of a unit in D / 64 parts by head dims and V in
// as many by positions (half as many per block of a pair, which holds half of
// the positions of K and half of the head dims of V), in the order of their use.
// K of a stage lies by 64 head dims, of all its positions each, as the product
// takes them at once; V page by page, as one box brings it: an instruction
// takes 16 positions of it, and no page is smaller.
//
// Bound (16 heads on 2 KV heads of 256 where nothing else is said; us in a graph,
// of the 6.79 TB/s and 1.93 PFLOP/s that a copy and a library product reach):
//   one token after 300 positions 10.5 us: two launches and a chain of trips to
//     memory of 0.7 us each (tables, page number, K, V, states, their merge);
//   one after 131,072 50 us, 5.4 TB/s; 64 sequences of 4096, 86 us, 6.3 TB/s: HBM;
//   a prompt of 4096 103 us, 1.34 PFLOP/s: the tiles' beginnings, ends and cuts;
//   2048 tokens after 16,384 307 to 338 us, a prompt of 16,384 1205 to 1235 us, 1.73 to
//     1.90 PFLOP/s, by the clock: the tensor cores;
//   2000 tokens after 28,000 positions, 16 heads on 4 of 128, 349 to 355 us, 1.36 PFLOP/s,
//     of 64 287 us: a unit's products are shorter than its softmax, and the issuing
//     warp has some 1200 cycles of its own per unit.
// Where two times are compared, here and below, both are of the step that chose
// between them, so the quicker one may be above what the call takes now.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kernels.h"
#include "kv8_attn.h"
#include "paged.cuh"
#include "tiles_ptx.cuh"

namespace bgmoe {
namespace paged {

using namespace tc;
using kv8::find_run;
using kv8::Place;
using kv8::seq_tiles;

constexpr int kRows = 128;  // rows of a block (TMEM lanes)
constexpr int kKeys = 128;  // positions of a unit
constexpr int kStages = 8;
constexpr int kStageBytes = 16384;
constexpr int kSoftWarps = 8, kAuxWarps = 4;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kLoadWarps = 2;
constexpr int kThreads = 512;
static_assert(kStages % kLoadWarps == 0, "a stage is one warp's");
constexpr int kMaxCtas = 256;  // workspace bound on the grid
// A run also pays for every tile it begins (Q, the first unit's chain, the
// output): the runs are cut on a scale where a tile with units takes some more
// places than units, before its first. A prompt of 4096 (16 heads on 2 x 256)
// takes 132, 114, 102, 103 us with 1, 2, 3, 5 of them, one of 40 heads on 8 x 128
// 190, 174, 168, 172; with few rows beginning and ending are cheap: with 0 to 3 a
// token of 64 sequences 36.3, 35.2, 36.7, 37.6, of 8 ragged ones 58.4, 55.3, 54.8, 54.7.
constexpr int kTileCost = 3, kFewRowsCost = 1;
constexpr float kMinusBig = -3.402823466e38f;  // running-max start, finite: m - m_new is never NaN
// Weights are 2^(x a - c), c = m a rounded (a: scale log2 e), where |c| is below
// this: c is off by up to 2^-17 there, which all weights that are made relative to one
// m share, but not those of another m: after a row's maximum moved, in the other half
// of a unit at 64 head dims, in another run's partial state. (Up to 2^20, where c is
// off by 2^-5, shares of a row's weight were wrong by up to 4 %.) Beyond it the
// other form costs 1 % in a prompt of 4096, 2 % of 2000 tokens after 28,000
// positions at 128 head dims, 3 % at 64.
constexpr float kLargeScore = 256.f;
// A row's scores may pass its m by this much (base 2: weights to 2^8) before O is
// scaled to a new one, but in calls of few rows (kByRowRows): there m is the
// largest score so far, whose weight is 1, so that where one position has most
// of a row its weight has no rounding. Decode waits for memory anyway (a token of
// 8 sequences of up to 65,536 55.6 us for 54.5); a prompt of 4096 takes 140 for 103.
constexpr float kSlack = 8.f;
constexpr int kByRowRows = 16;  // rows of a (sequence, KV head), on average, up to which a call is one of few rows
constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);  // A and B format in an instruction descriptor

template <int D, int kCtas>
struct Cfg {
  static constexpr int kTileRows = kRows * kCtas;     // MMA M
  static constexpr int kParts = D / 64 / kCtas;       // stages of a unit's K, and of its V
  static constexpr int kKeyRows = kKeys / kCtas;      // positions of K in a block ...
  static constexpr int kSlabsK = kCtas;               // ... in a stage, of 64 head dims each
  static constexpr int kDimsV = D / kCtas;            // head dims of V in a block ...
  static constexpr int kKeysV = kKeys / kParts;       // ... and positions of it in a stage
  static constexpr int kSlabsV = kDimsV / 64;
  static constexpr int kShiftK = kKeyRows == 128 ? 7 : 6, kShiftV = kKeysV == 128 ? 7 : kKeysV == 64 ? 6 : 5;
  static_assert((1 << kShiftK) == kKeyRows && (1 << kShiftV) == kKeysV, "shifts");
  // TMEM: O from column 0, then as many buffers of S as there is room for
  static constexpr bool kApart = D == 64;  // O of a unit's first half of positions, and of its second
  static constexpr int kBufs = D == 256 ? 2 : 3;
  static constexpr uint32_t kColS = 512 - 128 * kBufs;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kOutPitch = 144;               // bytes: 64 bf16 and padding
  static constexpr int kOutOffset = kQBytes + kStages * kStageBytes;
  static constexpr int kCtlOffset = kOutOffset + kSoftWarps * 16 * kOutPitch;
  static constexpr int kBytes = kCtlOffset + 4096 + 1024;  // + alignment slack
  static_assert(kKeyRows * kSlabsK * 128 == kStageBytes && kKeysV * kDimsV * 2 == kStageBytes, "stages");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Positions of a tile whose V is not finite, of those that not every row sees,
// as bits per unit from the first that has some. There are less than 257 of
// them (causal) or 513 (trees), so at most 6 units. Four tiles' bits: while
// the softmax ends tile t, V of t + 3 may come (S of t + 2 waits for the O of t
// + 1, which waits until O of t has been read); the MMA warp clears a tile's
// bits once its O has been read.
constexpr int kBadTiles = 4, kBadUnits = 8;
constexpr int kMaxBufs = 3;

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  // V of a unit that is to be looked through has come; it has been. The MMA
  // warp, which sees every phase of the stages, says the one and waits for the
  // other (a warp that skipped phases could take one for another).
  uint64_t look, fixed;
  uint64_t q_full, q_empty;
  uint64_t s_full[kMaxBufs], p_full[kMaxBufs];
  // One arrival per unit, on barriers in turn (Turn). A waiter's parity is safe if
  // it cannot be two phases off: the softmax of unit u has seen S of unit u,
  // whose commit covers the products of u - kBufs, and those from u on wait for
  // its weights.
  uint64_t pv_done[kMaxBufs];
  uint64_t o_empty;               // O of a finished tile has been read
  uint64_t peer_s[kMaxBufs], peer_o[kMaxBufs];  // the other block is ready for a unit's S, for its O
  uint64_t mx_full[4];            // both halves of a lane quadrant have stored their maxima (or sums)
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
  int bad_page;
  int bad_any[kBadTiles];
  uint32_t bad[kBadTiles][kBadUnits][kKeys / 32];
  float mx[2][2][kRows];  // [meetings in turn][half]
};

// Where a block's run starts, for the merge kernel: what every block of it reads
// of every run, and what it reads of the tiles that it joins.
struct __align__(8) RunHead {
  int tile;  // number of its first unit's tile
  int what;  // 0: no units; else 1, + 2 if it starts inside the tile, + 4 x the tile's rows
};
struct __align__(16) RunInfo {
  int g, rt, unused0, unused1;
  int lo, n, len, unused2;  // of its sequence
};

struct Params {
  const uint16_t* q;
  const int32_t* offsets;
  const int32_t* lens;
  const int32_t* tables;
  const unsigned long long* tree;  // null: causal
  uint16_t* o;
  float* part;    // two slots per run of [tile rows][D] O, then [tile rows] m and L
  RunHead* head;  // per run
  RunInfo* info;
  int32_t* flags;  // per block
  float scale_log2, slack;
  int B, T, Hq, Hkv, shift, n_pages, max_pages, words, q_stride;
  unsigned long long rmagic;  // ceil(2^36 / r), r = Hq / Hkv
  int cost;    // places of a tile beyond its units
  int by_row;  // few rows: layout of the partial states
  int narrow;  // find_small and find_tiles serve the call
  int stalled;
  long long timeout_ns;
};

// x / r for rows x < n r of n <= 2^24 tokens and r <= 64: with the magic off by
// less than r / r from 2^36 / r, x (magic - 2^36 / r) < 2^30 < 2^36 / r keeps the
// floor, and x magic < 2^24 (2^36 + r) stays in 64 bits.
__device__ __forceinline__ int div_r(int x, unsigned long long rmagic) {
  return (int)(((unsigned long long)(unsigned)x * rmagic) >> 36);
}

// kv8::tile_units without its division.
__device__ __forceinline__ int tile_units(const Params& p, int n, int len, int r, int RT, int rt) {
  const int see = len - n + div_r(min(n * r, (rt + 1) * RT) - 1, p.rmagic) + 1;
  return see > 0 ? (see + kKeys - 1) / kKeys : 0;
}

constexpr size_t slot_floats(int D, int tile_rows) { return (size_t)tile_rows * (D + 2); }

// Place in the run: unit i of the nb units of row tile rt of KV head g of
// sequence b. The roles go tile by tile (what a tile's units share is computed
// once: a warp of its own has 5 cycles for every instruction that it goes through).
struct Cursor {
  int b, g, rt, i, nb, n, len, lo;
  __device__ void sequence(const Params& p) {
    lo = ld(p.offsets + b);
    n = ld(p.offsets + b + 1) - lo;
    len = ld(p.lens + b);
  }
  // The next tile that has units.
  __device__ void next(const Params& p, int r, int RT) {
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
      nb = tile_units(p, n, len, r, RT, rt);
    } while (nb == 0);
  }
  // The tile's first position that some row does not see.
  __device__ int partial(const Params& p, int RT) const {
    return max(len - n + (p.tree != nullptr ? 0 : div_r(rt * RT, p.rmagic) + 1), 0);
  }
  // Units from the place on that every row sees all of. V of the others is looked through.
  __device__ int whole(const Params& p, int RT) const { return max(partial(p, RT) / kKeys - i, 0); }
};

// A buffer that is used in turn with others, and the phase of its barriers.
template <int kCount>
struct Turn {
  int at = 0;
  uint32_t phase = 0u;
  __device__ void next() {
    if (++at == kCount) at = 0, phase ^= 1u;
  }
};

// find_run for calls whose tables the block has in shared memory and whose sums
// the host knows to fit 32 bits (Params::narrow): the start of run c, by one
// warp. Every instruction here runs once, and cold, which is 5 to 10 cycles
// each; find_run's closed forms and 64-bit divisions are 1.6 us of a token's call
// and 5 of a prompt's.
//
// This one is for sequences of one row tile each (false: some have more). Lane k
// has `per` sequences from per k on.
constexpr int kSmall = 256;
__device__ __forceinline__ bool find_small(const Params& p, const int* offsets, const int* lens, int r, int RT, int cost,
                                           int c, int C, Place* out, bool* ok) {
  const int lane = threadIdx.x & 31, per = (p.B + 31) >> 5, b0 = lane * per, b1 = min(b0 + per, p.B);
  bool bad = false, wide = false;
  int v = 0, w = 0, t = 0;  // this lane's places, units, tiles, per KV head
  auto units_of = [&](int b) {  // the last row sees len positions
    return offsets[b + 1] > offsets[b] ? (lens[b] + kKeys - 1) / kKeys : 0;
  };
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int lo = offsets[b], hi = offsets[b + 1], len = lens[b];
    bad |= kv8::offsets_bad(lo, hi, b, p.B, p.T) || len < 0 || len > p.max_pages << p.shift;
    wide |= (hi - lo) * (long long)r > RT;
    const int nb = units_of(b);
    v += nb > 0 ? nb + cost : 0;
    w += nb;
    t += hi > lo;
  }
  *ok = !__any_sync(0xffffffffu, bad);
  if (!*ok) return true;
  if (__any_sync(0xffffffffu, wide)) return false;
  int vi = v, wi = w, ti = t;
#pragma unroll 1
  for (int o = 1; o < min(p.B, 32); o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, vi, o), y = __shfl_up_sync(0xffffffffu, wi, o);
    const int z = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) vi += x, wi += y, ti += z;
  }
  const int last = min(p.B, 32) - 1;  // the last lane that the sums reach
  const int N = __shfl_sync(0xffffffffu, vi, last) * p.Hkv, each = N / C, more = N - each * C;
  Place k{};
  k.b = -1;
  k.units = (long long)__shfl_sync(0xffffffffu, wi, last) * p.Hkv;
  const int from = c * each + min(c, more);
  const unsigned hit = __ballot_sync(0xffffffffu, vi * p.Hkv > from);
  if (hit != 0u) {  // (none: the end, all units are before it)
    const int L = __ffs(hit) - 1;
    // through lane L's sequences, by all lanes alike
    int off = from - __shfl_sync(0xffffffffu, vi - v, L) * p.Hkv, units = __shfl_sync(0xffffffffu, wi - w, L) * p.Hkv;
    int tiles = __shfl_sync(0xffffffffu, ti - t, L) * p.Hkv, b = L * per, nb = units_of(b);
    while (nb == 0 || off >= (nb + cost) * p.Hkv) {
      off -= nb > 0 ? (nb + cost) * p.Hkv : 0;
      units += nb * p.Hkv;
      tiles += offsets[b + 1] > offsets[b] ? p.Hkv : 0;
      nb = units_of(++b);
    }
    const int g = off / (nb + cost), i = max(off - g * (nb + cost) - cost, 0);
    k.b = b, k.g = g, k.rt = 0, k.i = i, k.nb = nb, k.tile = tiles + g;
    k.lo = offsets[b], k.n = offsets[b + 1] - k.lo, k.len = lens[b];
    k.units = units + g * nb + i;
  }
  *out = k;
  return true;
}

// The same for sequences of several tiles, up to kSmallTiles in all, which the warp
// goes through 32 at a time: first for every sequence's sums, then for the tile
// that the run starts in.
constexpr int kSmallTiles = 2048;
__device__ __forceinline__ void find_tiles(const Params& p, const int* offsets, const int* lens, int2* sums, int r, int RT,
                                           int cost, int c, int C, Place* out) {
  const int lane = threadIdx.x & 31;
  int N = 0, all_units = 0;
#pragma unroll 1
  for (int b = 0; b < p.B; ++b) {
    const int n = offsets[b + 1] - offsets[b], len = lens[b], tiles = seq_tiles(n, r, RT);
    int v = 0, w = 0;
#pragma unroll 1
    for (int rt = lane; rt < tiles; rt += 32) {
      const int nb = tile_units(p, n, len, r, RT, rt);
      v += nb > 0 ? nb + cost : 0;
      w += nb;
    }
    v = __reduce_add_sync(0xffffffffu, v);
    w = __reduce_add_sync(0xffffffffu, w);
    if (lane == 0) sums[b] = make_int2(v, w);
    N += v * p.Hkv;
    all_units += w * p.Hkv;
  }
  __syncwarp();
  const int each = N / C, more = N - each * C;
  Place k{};
  k.b = -1;
  k.units = all_units;
  int off = c * each + min(c, more);
  if (off < N) {  // (else the end: all units are before it)
    int b = 0, units = 0, tile = 0, n, len, tiles;
    int2 sum;
    while (true) {
      n = offsets[b + 1] - offsets[b], len = lens[b], tiles = seq_tiles(n, r, RT), sum = sums[b];
      if (off < sum.x * p.Hkv) break;
      off -= sum.x * p.Hkv, units += sum.y * p.Hkv, tile += tiles * p.Hkv;
      ++b;
    }
    const int g = off / sum.x;
    off -= g * sum.x, units += g * sum.y, tile += g * tiles;
    int nb, before, rt = 0;
    unsigned hit;
#pragma unroll 1
    while (true) {
      nb = rt + lane < tiles ? tile_units(p, n, len, r, RT, rt + lane) : 0;
      const int v = nb > 0 ? nb + cost : 0;
      int vi = v;
      before = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, vi, o), y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) vi += x, before += y;
      }
      before -= nb;
      hit = __ballot_sync(0xffffffffu, vi > off);
      const int at = hit != 0u ? __ffs(hit) - 1 : 31;
      if (hit != 0u) {
        off -= __shfl_sync(0xffffffffu, vi - v, at);
        break;
      }
      off -= __shfl_sync(0xffffffffu, vi, 31);
      units += __shfl_sync(0xffffffffu, before + nb, 31);
      rt += 32;
    }
    const int at = __ffs(hit) - 1, i = max(off - cost, 0);
    units += __shfl_sync(0xffffffffu, before, at) + i;
    k.b = b, k.g = g, k.rt = rt + at, k.i = i, k.nb = __shfl_sync(0xffffffffu, nb, at), k.tile = tile + rt + at;
    k.lo = offsets[b], k.n = n, k.len = len;
    k.units = units;
  }
  *out = k;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// What is left of a wait that outlasted a suspension: out of line, as it hardly
// ever runs and every wait has a call of it.
__device__ __noinline__ bool long_wait(uint64_t* bar, uint32_t parity, int* abort, long long timeout_ns) {
  return mbar_wait(bar, parity, abort, global_timer_ns() + (uint64_t)timeout_ns);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// *at |= bits in this block's and (of a pair) the other's shared memory, in
// front of what this thread releases after it.
template <int kCtas>
__device__ __forceinline__ void or_both(uint32_t* at, uint32_t bits, int rank) {
  atomicOr(at, bits);
  if (kCtas == 2) {
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n red.relaxed.cluster.shared::cluster.or.b32 [a], %2;\n}\n" ::
            "r"(smem_u32(at)),
        "r"(rank ^ 1), "r"(bits)
        : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
}

// Bits of the 64 positions from `first` on that the tree lets a draft see,
// whose words are at w: all of the context's (before ctx), then its own.
__device__ __forceinline__ uint64_t tree_bits(const unsigned long long* w, int words, int first, int ctx) {
  const int j = first - ctx;
  if (j <= -64) return ~0ull;
  if (j < 0) return (ld(w) << -j) | ((1ull << -j) - 1);
  const int k = j >> 6, s = j & 63;
  uint64_t v = k < words ? ld(w + k) >> s : 0ull;
  if (s > 0 && k + 1 < words) v |= ld(w + k + 1) << (64 - s);
  return v;
}

// 1 / l of a row, whose sum of weights l is 0 in two cases: it sees nothing, and is
// zero; or all that it sees scores -inf, and its softmax is NaN. ctx: positions
// before the new ones; token: of the call, the tok-th of its sequence.
__device__ __noinline__ float inverse_of_none(const unsigned long long* tree, int words, int token, int tok, int ctx) {
  const int see = ctx + tok + 1;
  bool any = see > 0 && (tree == nullptr || ctx > 0);
  if (!any && see > 0) {
#pragma unroll 1
    for (int first = 0; first < see && !any; first += 64) {
      const uint64_t bits = tree_bits(tree + (size_t)token * words, words, first, ctx);
      any = (see - first >= 64 ? bits : bits & ((1ull << (see - first)) - 1)) != 0ull;
    }
  }
  return any ? __uint_as_float(0x7FC00000u) : 0.f;
}

template <int D, int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const Params p) {
  using F = Cfg<D, kCtas>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;               // 64-dim slabs of 128 rows x 128 bytes
  uint8_t* sR = smem + F::kQBytes;  // the ring
  constexpr int kTileRows = F::kTileRows, kBufs = F::kBufs;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + F::kCtlOffset);
  static_assert(sizeof(Ctl) <= 4096, "control block");
  __shared__ long long s_unit[2];  // units before the run's start and end
  __shared__ Cursor s_cur;
  __shared__ int s_bad, s_tile;
  __shared__ int s_offsets[kSmall + 1], s_lens[kSmall];
  __shared__ int2 s_sums[2][kSmall];

  // The warp's number through a shuffle, which the compiler knows to be
  // uniform: the roles' loops then run on uniform registers, where the MMA
  // instructions take their descriptors from.
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int C = gridDim.x / kCtas, c = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;  // runs, run, block of its tiles
  const int r = p.Hq / p.Hkv;

  if (threadIdx.x == 32) {
    mbar_init(&ctl->q_full, kAuxWarps);
    mbar_init(&ctl->q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int i = 0; i < kMaxBufs; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], kSoftWarps);
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->peer_s[i], 1);
      mbar_init(&ctl->peer_o[i], 1);
    }
    mbar_init(&ctl->o_empty, kSoftWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&ctl->mx_full[i], 2);
    mbar_init(&ctl->look, 1);
    mbar_init(&ctl->fixed, kAuxWarps);
    mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    ctl->bad_page = 0;
    fence_barrier_init();
  }
  if (warp == kAuxWarps + kSoftWarps - 1) {
    uint32_t* z = &ctl->bad[0][0][0];
    for (int i = lane; i < kBadTiles * kBadUnits * (kKeys / 32); i += 32) z[i] = 0u;
    if (lane < kBadTiles) ctl->bad_any[lane] = 0;
  }
  if (warp == kMmaWarp) alloc_columns<kCtas>(&ctl->tmem);
  if (warp == kLoadWarp && lane < 2) prefetch_tmap(lane == 0 ? &tm_k : &tm_v);
  // (the other block's barriers and columns are waited for when they are needed)
  if (kCtas == 2) {
    tc_fence_before();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  }
  // Launched with programmatic dependent launch: wait for the kernels before
  // this one, then let this call's merge launch (it waits in turn). A block that
  // waits here holds its columns, but those it waits for have theirs: they all
  // run, or have ended, before it starts.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.narrow) {
    if (threadIdx.x <= p.B) s_offsets[threadIdx.x] = ld(p.offsets + threadIdx.x);
    if (threadIdx.x < p.B) s_lens[threadIdx.x] = ld(p.lens + threadIdx.x);
    __syncthreads();
  }
  if (warp == 1 || warp == 2) {  // the run's start and its end
    Place k;
    bool ok = true;
    const int at = c + warp - 1;
    if (!p.narrow)
      ok = find_run(p.offsets, p.lens, p.B, p.T, p.Hkv, p.max_pages << p.shift, r, kTileRows, kKeys, p.cost, at, C, &k);
    else if (!find_small(p, s_offsets, s_lens, r, kTileRows, p.cost, at, C, &k, &ok))
      find_tiles(p, s_offsets, s_lens, s_sums[warp - 1], r, kTileRows, p.cost, at, C, &k);
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
  int wide = 0;  // a sequence has more drafts than its words have bits
  if (p.tree != nullptr && warp > 2)
    for (int b = threadIdx.x - 96; b < p.B; b += kThreads - 96)
      wide |= ld(p.offsets + b + 1) - ld(p.offsets + b) > 64 * p.words;
  if (__syncthreads_or(wide)) {
    if (threadIdx.x == 0) s_bad = 1;
    __syncthreads();
  }
  const bool idle = s_bad || s_unit[0] >= s_unit[1];  // both blocks of a run alike
  // A lane's page of the w-th 32 of a sequence, as the table has it; anything past the context.
  // (Whether it is there, and needed, is asked where it is used: the value is on its way until then.)
  auto look_up = [&](const Cursor& k, int w) -> int {
    const int page = 32 * w + lane;
    return page << p.shift < k.len ? ld(p.tables + (size_t)k.b * p.max_pages + page) : 0;
  };
  const bool loads = warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps;
  const int first_window = s_cur.i * kKeys >> p.shift >> 5;
  const int first_pages = loads && !idle ? look_up(s_cur, first_window) : 0;  // on their way meanwhile
  if (kCtas == 2) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  } else {
    tc_fence_before();
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  if (threadIdx.x == 0) {
    const bool live = !s_bad && s_unit[0] < s_unit[1];
    if (rank == 0) {
      const int there = min(kTileRows, s_cur.n * r - s_cur.rt * kTileRows);
      p.head[c] = RunHead{s_tile, live ? 1 + (s_cur.i > 0 ? 2 : 0) + 4 * there : 0};
      p.info[c] = RunInfo{s_cur.g, s_cur.rt, 0, 0, s_cur.lo, s_cur.n, s_cur.len, 0};
    }
    if (!live) p.flags[blockIdx.x] = s_bad ? (int32_t)MOE_ERR_INVALID_ARG : 0;
  }
  // Queries that see nothing (more queries than positions): o = 0.
  for (int b = blockIdx.x; !s_bad && b < p.B; b += gridDim.x) {
    const int lo = ld(p.offsets + b), hi = ld(p.offsets + b + 1), len = ld(p.lens + b);
    const size_t pieces = (size_t)max(0, hi - lo - len) * p.Hq * (D / 8);
    uint4* z = reinterpret_cast<uint4*>(p.o + (size_t)lo * p.Hq * D);
    for (size_t i = threadIdx.x; i < pieces; i += kThreads) z[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (idle) {
    tile_barrier<kCtas>();  // (columns of a pair are freed by both)
    if (warp == kMmaWarp) free_columns<kCtas>(tmem);
    return;
  }
  const int U = (int)(s_unit[1] - s_unit[0]);
  Cursor cur = s_cur;

  // Each wait has its own limit (a long call may run for longer than one), set
  // only once it has lasted for a suspension (up to 0.5 ms) already.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity);
    if (!ok) ok = long_wait(bar, parity, &ctl->abort, p.timeout_ns);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  // Stage h of the block at a place of the ring, and its phase there.
  auto stage = [](int place, int h) { return (place * F::kParts + h) % kStages; };
  auto phase = [](int place, int h) { return (uint32_t)((place * F::kParts + h) / kStages) & 1u; };

  if (warp == kMmaWarp) {
    // ------------------------------------------------------- MMA issuer
    // With two blocks the leader's warp issues for both; the other's goes
    // through the same steps, waits for what its own block has to have ready
    // and passes that on as one arrival.
    constexpr uint32_t idesc_s = idesc_f16_f32(kTileRows, kKeys) | kBf16;
    constexpr uint32_t idesc_o = idesc_f16_f32(kTileRows, D) | kBf16 | (1u << 16);  // B is MN-major
    const uint64_t dq = sw128_desc(smem_u32(sQ));
    const uint32_t leader = elect_one();
    const uint64_t dk = sw128_desc(smem_u32(sR));
    // V of a stage lies page by page (or its part of one), of each the 64 head dims
    // side by side
    const int vs = min(p.shift, F::kShiftV);  // positions of a box, as a shift
    const uint64_t dv = sw128_mn_desc(smem_u32(sR), 128u << vs);
    int tq = 0, to = 0;     // tiles whose Q has been waited for, whose O has been started
    uint32_t fixes = 0u;    // units whose V was looked through
    int place = 0;          // in the ring, in units of a K or V block
    Turn<kBufs> sb, ob;     // S of the unit to be scored, of that to be put out
    Cursor nxt = cur;
    // Waits until a step of a unit may begin: its stages, the softmax's or Q's
    // barrier `own` (if any), the other block's arrival; all tested together.
    // The other block's warp passes its readiness on. (An arrival for unit u +
    // kBufs comes after the leader's step of unit u: as many barriers in turn will do.)
    bool there = false;  // all stages of the step are
    auto ready = [&](uint64_t* own, uint32_t parity, uint64_t* peer, uint32_t peer_parity, bool fixed) -> bool {
      bool all = own == nullptr || mbar_test_wait(own, parity);
#pragma unroll
      for (int h = 0; h < F::kParts; ++h) all = mbar_test_wait(&ctl->full[stage(place, h)], phase(place, h)) && all;
      const bool listens = kCtas == 2 && rank == 0;
      if (listens) all = test_cluster(peer, peer_parity) && all;
      there = __all_sync(0xffffffffu, all);
      if (fixed || !there) {
        // (a block on its own takes its stages one by one, as they come: part())
        for (int h = 0; (kCtas == 2 || fixed) && h < F::kParts; ++h)
          if (!warp_wait(&ctl->full[stage(place, h)], phase(place, h))) return false;
        if (fixed && lane == 0) mbar_arrive(&ctl->look);
        if (own != nullptr && !warp_wait(own, parity)) return false;
        if (fixed && !warp_wait(&ctl->fixed, fixes++ & 1u)) return false;
        if (listens && !warp_wait(peer, peer_parity)) return false;
        // (a test at cluster scope, for the fence below to follow on)
        if (listens && !__all_sync(0xffffffffu, test_cluster(peer, peer_parity))) return false;
      }
      tc_fence_after();
      if (listens) acquire_peer();
      if (kCtas == 2 && rank != 0) {
        tc_fence_before();
        if (lane == 0) arrive_leader(peer);
      }
      return true;
    };
    auto part = [&](int h) { return kCtas == 2 || there || warp_wait(&ctl->full[stage(place, h)], phase(place, h)); };
    auto score = [&](bool first, bool ends) -> bool {  // S of the next unit
      const int buf = sb.at;
      if (!ready(first ? &ctl->q_full : nullptr, tq & 1, &ctl->peer_s[buf], sb.phase, false)) return false;
      sb.next();
      tq += first;
      if (rank != 0) return true;
      const uint32_t d = tmem + F::kColS + 128 * buf;
#pragma unroll
      for (int h = 0; h < F::kParts; ++h) {
        const int st = stage(place, h);
        if (!part(h)) return false;
#pragma unroll
        for (int kk = 0; kk < 4 * F::kSlabsK; ++kk) {
          const uint32_t slab = kk >> 2, in = (kk & 3) * 2;  // 64-dim slabs
          mma_ss<kCtas>(d, dq + (h * F::kSlabsK + slab) * (kRows * 128 / 16) + in,
                        dk + st * (kStageBytes / 16) + slab * (F::kKeyRows * 128 / 16) + in, idesc_s, kk > 0 || h > 0,
                        leader);
        }
        commit<kCtas>(&ctl->empty[st], leader);
      }
      commit<kCtas>(&ctl->s_full[buf], leader);
      if (ends) commit<kCtas>(&ctl->q_empty, leader);
      return true;
    };
    auto output = [&](bool first, bool fix) -> bool {  // O of the next
      if (first && to++ > 0) {
        if (!warp_wait(&ctl->o_empty, (to - 2) & 1)) return false;
        const int t = (to - 2) % kBadTiles;
        if (ctl->bad_any[t]) {
          for (int i = lane; i < kBadUnits * (kKeys / 32); i += 32) (&ctl->bad[t][0][0])[i] = 0u;
          __syncwarp();
          if (lane == 0) ctl->bad_any[t] = 0;
          __syncwarp();
        }
      }
      const int buf = ob.at;
      if (!ready(&ctl->p_full[buf], ob.phase, &ctl->peer_o[buf], ob.phase, fix)) return false;
      ob.next();
      if (rank != 0) return true;
      const uint32_t a = tmem + F::kColS + 128 * buf;
#pragma unroll
      for (int h = 0; h < F::kParts; ++h) {
        const int st = stage(place, h);
        if (!part(h)) return false;
#pragma unroll
        for (int kk = 0; kk < F::kKeysV / 16; ++kk) {
          const int key = h * F::kKeysV + kk * 16, second = F::kApart && key >= 64;
          mma_ts<kCtas>(tmem + second * D, a + key / 2 + 32 * second,
                        dv + st * (kStageBytes / 16) +
                            ((((kk * 16) >> vs) * F::kSlabsV << (vs + 3)) + (((kk * 16) & ((1 << vs) - 1)) << 3)),
                        idesc_o, key > 64 * second ? 1u : (uint32_t)!first, leader);
        }
        commit<kCtas>(&ctl->empty[st], leader);
      }
      commit<kCtas>(&ctl->pv_done[buf], leader);
      return true;
    };
    // S goes ahead of O of a unit, whose weights the softmax makes meanwhile, as
    // far as there are buffers; not over a tile's end: the next one's Q may be
    // long in coming. (One call site each: the code stays short.)
    bool ok = true;
#pragma unroll 1
    for (int u = 0, nu; ok && u < U; u += nu) {
      nu = min(nxt.nb - nxt.i, U - u);
      const int whole = nxt.whole(p, kTileRows);
#pragma unroll 1
      for (int j = 1 - kBufs; ok && j < nu; ++j) {
        const int e = j + kBufs - 1;
        if (e < nu) {
          ok = score(e == 0, e == nu - 1);
          ++place;
        }
        if (ok && j >= 0) {
          ok = output(j == 0, j >= whole);
          ++place;
        }
      }
      if (u + nu < U) nxt.next(p, r, kTileRows);
    }
    if (rank == 0) commit<kCtas>(&ctl->mma_done, leader);
  } else if (loads) {
    // ---------------------------------------------------- K and V by TMA
    const int outside = p.n_pages * p.Hkv;  // a page that reads as zeros
    const int rows = 1 << p.shift;
    const bool many = rows < kKeys;  // a unit has several pages
    // This lane's box of a stage: of V all of the stage's head dims of a page's
    // positions, as of K where a page holds all of the stage's positions, else 64
    // (a product takes all positions of K at once, but 16 of V).
    struct Box {
      int key, slab, to;  // its first position and 64 head dims, its place in the stage
      bool on;
      __device__ Box(int page_shift, int keys_shift, int slabs, bool whole, int key0, int slab0) {
        const int box_shift = min(page_shift, keys_shift), per_shift = keys_shift - box_shift;
        const int lane = threadIdx.x & 31, s = lane >> per_shift, n = lane & ((1 << per_shift) - 1);
        on = s < (whole || per_shift == 0 ? 1 : slabs);
        key = key0 + (n << box_shift);
        slab = slab0 + s;
        to = whole ? (n * slabs) << (box_shift + 7) : (s << (keys_shift + 7)) + (n << (box_shift + 7));
      }
    };
    const Box bk(p.shift, F::kShiftK, F::kSlabsK, false, rank * F::kKeyRows, 0);
    const Box bv(p.shift, F::kShiftV, F::kSlabsV, true, 0, rank * F::kSlabsV);
    int issued = 0;
    bool bad = false;
    auto settle = [&](int id, int g, bool needed) -> int {  // its place in the pools
      const bool there = id >= 0 && id < p.n_pages;
      bad |= needed && !there;
      return needed && there ? id * p.Hkv + g : outside;
    };
    if ((int)blockIdx.x != p.stalled) {
      // K and V of every unit in the order of their use, one copy of the code:
      // it runs cold. The warps go through the same steps, and each fills the stages
      // that are its own (and so sees every phase of their barriers: one that did
      // not could take one for another).
      Cursor k = cur;
      int window = first_window;                            // 32 of the sequence's pages, in the lanes ...
      int pages = first_pages, then = look_up(k, window + 1);  // ... and the 32 after them
      int z[kBufs] = {};  // pages of the units whose V is to come, of the last K's
      int place = 0;
      bool ok = true;
#pragma unroll 1
      for (int u = 0, nu; ok && u < U; u += nu) {
        const int i0 = k.i;
        nu = min(k.nb - i0, U - u);
#pragma unroll 1
        for (int j = 1 - kBufs; ok && j < nu; ++j) {
          const int e = j + kBufs - 1;
#pragma unroll
          for (int i = 0; i + 1 < kBufs; ++i) z[i] = z[i + 1];
          if (e < nu) {
            const int page = (i0 + e) * kKeys >> p.shift;
            if (page >> 5 != window) {
              pages = then;
              then = look_up(k, ++window + 1);
            }
            const int id = __shfl_sync(0xffffffffu, pages, page + lane);
            // the unit's, as far as the context goes
            z[kBufs - 1] = settle(id, k.g, (lane == 0 || lane << p.shift < kKeys) && (page + lane) << p.shift < k.len);
          }
#pragma unroll 1
          for (int v = e < nu ? 0 : 1; ok && v < (j < 0 ? 1 : 2); ++v, ++place) {
            const bool is_k = v == 0;
            const int first = (i0 + (is_k ? e : j)) * kKeys, at_page = is_k ? z[kBufs - 1] : z[0];
            const CUtensorMap* map = is_k ? &tm_k : &tm_v;
            const int to = is_k ? bk.to : bv.to;
            const bool on = is_k ? bk.on : bv.on;
            int key = is_k ? bk.key : bv.key, slab = is_k ? bk.slab : bv.slab;
#pragma unroll 1
            for (int h = 0; h < F::kParts; ++h) {
              if (stage(place, h) % kLoadWarps == warp - kLoadWarp) {
                const int st = stage(place, h);
                ok = warp_wait(&ctl->empty[st], phase(place, h) ^ 1u);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], kStageBytes);
                const int at = __shfl_sync(0xffffffffu, at_page, many ? (key >> p.shift) & 31 : 0);
                if (on) tma_load_4d(sR + st * kStageBytes + to, map, 0, (first + key) & (rows - 1), slab, at, &ctl->full[st]);
                issued = place * F::kParts + h + 1;
              }
              if (is_k) slab += F::kSlabsK;
              else key += F::kKeysV;
            }
            if (is_k && e + 1 == nu && u + nu < U) {  // the next tile's pages come while this unit's V waits for room
              k.next(p, r, kTileRows);
              window = 0;
              pages = look_up(k, 0);
              then = look_up(k, 1);
            }
          }
        }
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) ctl->bad_page = 1;
    // No copy may be in flight when the block ends, whatever ended the loops.
    int dummy = 0;
    for (int j = issued - 1; j >= max(issued - kStages, 0); j -= kLoadWarps)  // its own
      mbar_wait(&ctl->full[j % kStages], (uint32_t)(j / kStages) & 1u, &dummy,
                global_timer_ns() + (uint64_t)kv8::kTimeoutNs);
  } else if (warp < kSoftWarps) {
    // --------------------------------------------------------- softmax
    const int quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    // (with any a > 0 and m >= kMinusBig: what is not seen, -inf, weighs 0, and a row that has seen
    // nothing yet has L = 0 and O = 0, whatever factor they take)
    const float a = p.scale_log2;
    constexpr int kOwn = F::kApart ? D : D / 2;  // columns of O that a half scales
    int met = 0;
    // This thread's value and its partner's, once both are there. At 128 head dims,
    // where the softmax bounds, by a barrier of the two warps alone (2000 tokens
    // after 28,000 positions 349 us for 362; at 256 a prompt of 4096 takes 104 for
    // 102.5 so). It has no limit of its own: either warp comes there, or gives up
    // within the limits of its other waits, has said so by then, and arrives once
    // in passing (below).
    constexpr bool kAlone = D == 128;
    auto meet = [&](float v, float& other) -> bool {
      ctl->mx[met & 1][half][row] = v;
      if constexpr (kAlone) {
        asm volatile("barrier.sync.aligned %0, 64;" ::"r"(1 + quad) : "memory");
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->mx_full[quad]);
        if (!warp_wait(&ctl->mx_full[quad], met & 1)) return false;
      }
      other = ctl->mx[met & 1][half ^ 1][row];
      ++met;
      return !kAlone || __all_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&ctl->abort) == 0);
    };
    Cursor un = cur;
    Turn<kBufs> sb;  // the unit's S, P and barriers
    bool ok = true;
#pragma unroll 1
    for (int u = 0, nu, tile = 0; ok && u < U; u += nu, ++tile) {
      nu = min(un.nb - un.i, U - u);
      const int whole = un.whole(p, kTileRows);
      const int rho = un.rt * kTileRows + rank * kRows + row, tok = div_r(rho, p.rmagic);
      const int see = rho < un.n * r ? max(un.len - un.n + tok + 1, 0) : 0;
      const bool act = __any_sync(0xffffffffu, see > 0);  // some row of the warp's is there
      float m = kMinusBig, l = 0.f, f0 = 1.f, f1 = 1.f;
      const int ctx = un.len - un.n;  // positions before the new ones
      float other;
#pragma unroll 1
      for (int j = 0; j < nu; ++j) {
        ok = warp_wait(&ctl->s_full[sb.at], sb.phase);
        if (!ok) break;
        if (act) {
          tc_fence_after();
          const uint32_t ts = lane_addr + F::kColS + 128 * sb.at;
          uint32_t x[64];
          tmem_ld_64(ts + 64 * half, x);
          if (j >= whole) {
            const int first = (un.i + j) * kKeys + 64 * half;
            // Rows that are not there, or see nothing, are left to themselves: nothing
            // of theirs is written, and a warp may have one row and 31 such.
            const int left = see > 0 ? see - first : kKeys;  // visible positions from this half's first on (but for the tree)
            if (__any_sync(0xffffffffu, left < 64 || (p.tree != nullptr && first + 64 > ctx))) {
              uint64_t bits = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0ull;
              if (p.tree != nullptr && see > 0)
                bits &= tree_bits(p.tree + (size_t)(un.lo + tok) * p.words, p.words, first, ctx);
              const uint32_t b0 = (uint32_t)bits, b1 = (uint32_t)(bits >> 32);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (!(b0 >> e & 1u)) x[e] = 0xFF800000u;  // -inf
                if (!(b1 >> e & 1u)) x[32 + e] = 0xFF800000u;
              }
            }
          }
          float mx = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
          for (int e = 2; e < 64; e += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
          if (!F::kApart) {
            ok = meet(mx, other);
            if (!ok) break;
            mx = fmaxf(mx, other);
          }
          if (j == 0) {
            m = fmaxf(mx, kMinusBig);
          } else if (__any_sync(0xffffffffu, see > 0 && (mx - m) * a > p.slack)) {
            // O and L to the new maximum, once the products of the last unit are in
            const float nm = see > 0 && (mx - m) * a > p.slack ? mx : m, f = ex2((m - nm) * a);
            m = nm;
            l *= f;
            ok = warp_wait(&ctl->pv_done[sb.at > 0 ? sb.at - 1 : kBufs - 1], sb.at > 0 ? sb.phase : sb.phase ^ 1u);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int d = half * kOwn; d < (half + 1) * kOwn; d += 16) {
              uint32_t w[16];
              tmem_ld_16(lane_addr + d, w);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
              tmem_st_16(lane_addr + d, w);
            }
          }
          // weights, over S (apart, over what this half has read, else over the first half, which
          // both have read)
          auto weights = [&](auto step) {  // 2^step(two values)
            uint64_t s2 = 0ull;
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const float2 y = unpack2(step(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]))));
              const float w0 = ex2(y.x), w1 = ex2(y.y);
              s2 = add2(s2, pack2(w0, w1));
              w[e / 2] = pack_bf16(w0, w1);
            }
            const float2 s = unpack2(s2);
            l += s.x + s.y;
            tmem_st_32(ts + (F::kApart ? 64 : 32) * half, w);
          };
          const uint64_t a2 = pack2(a, a);
          const float c = m * a;
          if (!__any_sync(0xffffffffu, see > 0 && !(fabsf(c) < kLargeScore))) {
            // x a - c in one step
            const uint64_t c2 = pack2(-c, -c);
            weights([&](uint64_t v) { return fma2(v, a2, c2); });
          } else {  // the difference first: off by 2^-24 of itself
            const uint64_t m2 = pack2(-m, -m);
            weights([&](uint64_t v) { return mul2(add2(v, m2), a2); });
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[sb.at]);
        if (j + 1 < nu) sb.next();
      }
      if (!ok) break;
      // ---- the run leaves this tile: its rows' outputs, or the partial state
      const bool mid = un.i > 0, ends = un.i + nu == un.nb;  // began in an earlier run; ends in this one
      if (act) {
        ok = meet(l, other);
        if (!ok) break;
        if (F::kApart) {  // the two halves' states as one
          const float l0 = half == 0 ? l : other, l1 = half == 0 ? other : l;
          ok = meet(m, other);
          if (!ok) break;
          const float m0 = half == 0 ? m : other, m1 = half == 0 ? other : m;
          m = fmaxf(m0, m1);
          f0 = ex2((m0 - m) * a);
          f1 = ex2((m1 - m) * a);
          l = l0 * f0 + l1 * f1;
        } else {
          l += other;
        }
      }
      ok = warp_wait(&ctl->pv_done[sb.at], sb.phase);
      if (!ok) break;
      sb.next();
      tc_fence_after();
      if (act) {
        const int bt = tile % kBadTiles;
        if (ctl->bad_any[bt]) {
          // a row that sees one of these is NaN, as its products would have made it
          const int b0 = max(ctx + (p.tree != nullptr ? 0 : div_r(un.rt * kTileRows, p.rmagic) + 1), 0) / kKeys;
          for (int q = 0; q < kBadUnits * (kKeys / 32); ++q) {
            uint32_t bits = (&ctl->bad[bt][0][0])[q];
            const int pos = b0 * kKeys + 32 * q;
            if (bits == 0u || see <= pos) continue;
            if (see - pos < 32) bits &= (1u << (see - pos)) - 1u;
            if (p.tree != nullptr)
              bits &= (uint32_t)tree_bits(p.tree + (size_t)(un.lo + tok) * p.words, p.words, pos, ctx);
            if (bits != 0u) l = __uint_as_float(0x7FC00000u);
          }
        }
        const int d0 = half * (D / 2);
        const uint32_t out = smem_u32(smem + F::kOutOffset) + warp * (16 * F::kOutPitch);
        if (!mid && ends) {
          float inv = 1.f / l;
          if (l == 0.f) inv = see > 0 ? inverse_of_none(p.tree, p.words, un.lo + tok, tok, ctx) : 0.f;
          f0 *= inv, f1 *= inv;
          // 16 rows by 64 dims at a time through shared memory: 8 lanes write a row's
          // 128 bytes, 4 rows at once. A half has half of the dims of all rows, or
          // all dims of half of them. (32 rows by 32 dims, whose stores write half
          // lines: a prompt of 4096 106.9 us for 104.3, without the stores 101.9.)
#pragma unroll 1
          for (int i = D == 64 ? half : 0; i < (D == 64 ? half + 1 : 2); ++i) {
            uint16_t* orow[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rk = un.rt * kTileRows + rank * kRows + quad * 32 + 16 * i + 4 * k + (lane >> 3);
              const int tk = div_r(rk, p.rmagic);
              const bool live = rk < un.n * r && ctx + tk >= 0;
              uint16_t* at = p.o + ((size_t)(un.lo + tk) * p.Hq + (size_t)un.g * r + rk - tk * r) * D + 8 * (lane & 7);
              orow[k] = live ? at : nullptr;
            }
#pragma unroll 1
            for (int j = D == 64 ? 0 : d0; j < (D == 64 ? D : d0 + D / 2); j += 64) {
              __syncwarp();
#pragma unroll
              for (int h = 0; h < 64; h += 32) {
                float v[32];
                tmem_ld_32(lane_addr + j + h, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= f0;
                if (F::kApart) {
                  float w[32];
                  tmem_ld_32(lane_addr + D + j + h, w);
#pragma unroll
                  for (int e = 0; e < 32; ++e) v[e] = fmaf(w[e], f1, v[e]);
                }
                if ((lane >> 4) == i) {
#pragma unroll
                  for (int e = 0; e < 32; e += 8)
                    sts128(out + (lane & 15) * F::kOutPitch + 2 * (h + e), pack_bf16(v[e], v[e + 1]),
                           pack_bf16(v[e + 2], v[e + 3]), pack_bf16(v[e + 4], v[e + 5]), pack_bf16(v[e + 6], v[e + 7]));
                }
              }
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 y = lds128(out + (4 * k + (lane >> 3)) * F::kOutPitch + 16 * (lane & 7));
                if (orow[k]) *reinterpret_cast<uint4*>(orow[k] + j) = y;
              }
            }
          }
        } else {
          float* part = p.part + (size_t)(2 * c + (mid ? 0 : 1)) * slot_floats(D, kTileRows);
          // row by row, or 4 head dims of all rows side by side
          const size_t step = p.by_row ? 1 : kTileRows;
          float4* to = reinterpret_cast<float4*>(part) + (p.by_row ? (size_t)(rank * kRows + row) * (D / 4) + d0 / 4
                                                                   : (size_t)(d0 / 4) * kTileRows + rank * kRows + row);
          const bool there = un.rt * kTileRows + rank * kRows + row < un.n * r;
#pragma unroll 1
          for (int j = 0; j < D / 2; j += 32) {
            float v[32];
            tmem_ld_32(lane_addr + d0 + j, v);
            if (F::kApart) {
              float w[32];
              tmem_ld_32(lane_addr + D + d0 + j, w);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = fmaf(w[e], f1, v[e] * f0);
            }
            if (there) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[e * step] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
            to += 8 * step;
          }
          if (half == 0 && there) {
            part[(size_t)D * kTileRows + rank * kRows + row] = m;
            part[(size_t)(D + 1) * kTileRows + rank * kRows + row] = l;
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_empty);
      if (u + nu < U) un.next(p, r, kTileRows);
    }
    if (kAlone && !ok) asm volatile("barrier.arrive.aligned %0, 64;" ::"r"(1 + quad) : "memory");
  } else if (warp < kSoftWarps + kAuxWarps) {
    // ------------------------------------------- Q, and V that is not finite
    const int t = threadIdx.x - 32 * kSoftWarps;
    constexpr int kThr = 32 * kAuxWarps, kLanes = D / 8, kAtOnce = kThr / kLanes;  // lanes per row, rows per step
    const int ln = t % kLanes, row0 = t / kLanes;
    const uint32_t q0 = smem_u32(sQ) + (ln >> 3) * (kRows * 128);
    Cursor k = cur;
    bool ok = true;
    uint32_t fixes = 0u;
#pragma unroll 1
    for (int u = 0, nu, tile = 0; ok && u < U; u += nu, ++tile) {
      nu = min(k.nb - k.i, U - u);
      if (tile > 0 && !warp_wait(&ctl->q_empty, (tile - 1) & 1)) break;
      tc_fence_after();
      const int rho0 = k.rt * kTileRows + rank * kRows, rows = min(kRows, k.n * r - rho0);
#pragma unroll 4
      for (int i = row0; i < rows; i += kAtOnce) {
        const int rho = rho0 + i, tok = div_r(rho, p.rmagic);
        const uint16_t* from = p.q + (size_t)(k.lo + tok) * p.q_stride + (size_t)(k.g * r + rho - tok * r) * D + ln * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(q0 + i * 128 + (((ln & 7) ^ (i & 7)) << 4)),
                     "l"(from)
                     : "memory");
      }
      cp_async_wait_all();
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full);
      const int part = k.partial(p, kTileRows), bt = tile % kBadTiles;
#pragma unroll 1
      for (int j = k.whole(p, kTileRows); ok && j < nu; ++j) {
        // in the ring V of unit u + j comes after K of so many units
        const int place = 2 * (u + j) + 1 + min(kBufs - 1, nu - 1 - j), first = (k.i + j) * kKeys;
        ok = warp_wait(&ctl->look, fixes & 1u);
        if (!ok) break;
        const int vs = min(p.shift, F::kShiftV);
#pragma unroll 1
        for (int h = 0; ok && h < F::kParts; ++h) {
          const int st = stage(place, h);
          ok = warp_wait(&ctl->full[st], phase(place, h));
          if (!ok) break;
          const int key0 = max(part - first - h * F::kKeysV, 0);
          const uint32_t base = smem_u32(sR) + st * kStageBytes;
          // in the order in which the stage lies, from key0's page on
          const int i0 = ((key0 >> vs) * (8 * F::kSlabsV) << vs) + t;
          uint32_t odd = 0u;
#pragma unroll 4
          for (int i = i0; i < kStageBytes / 16; i += kThr) {
            const uint4 v = lds128(base + 16 * i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= (w[e] & 0x7F807F80u) + 0x00800080u;  // bits 15, 31: an exponent of ones
          }
          if (!__any_sync(0xffffffffu, odd & 0x80008000u)) continue;
#pragma unroll 1
          for (int i = i0; i < kStageBytes / 16; i += kThr) {
            const int key = (((i >> (3 + vs)) / F::kSlabsV) << vs) + ((i >> 3) & ((1 << vs) - 1));
            const uint4 v = lds128(base + 16 * i);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7F80u) == 0x7F80u) {
                w[e] &= 0xFFFF0000u;
                found = true;
              }
              if ((w[e] & 0x7F800000u) == 0x7F800000u) {
                w[e] &= 0xFFFFu;
                found = true;
              }
            }
            if (!found || key < key0) continue;
            sts128(base + 16 * i, w[0], w[1], w[2], w[3]);
            if (first + h * F::kKeysV + key >= k.len) continue;  // (what lies behind the context is nobody's)
            const int bu = k.i + j - part / kKeys, key_u = h * F::kKeysV + key;
            or_both<kCtas>(&ctl->bad[bt][bu][key_u >> 5], 1u << (key_u & 31), rank);
            or_both<kCtas>(reinterpret_cast<uint32_t*>(&ctl->bad_any[bt]), 1u, rank);
          }
        }
        if (!ok) break;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->fixed);
        ++fixes;
      }
      if (u + nu < U) k.next(p, r, kTileRows);
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
  if (threadIdx.x == 0)
    p.flags[blockIdx.x] = *reinterpret_cast<volatile int*>(&ctl->abort) ? (int32_t)MOE_ERR_DEVICE_TIMEOUT
                          : ctl->bad_page ? (int32_t)MOE_ERR_INVALID_ARG
                                          : 0;
}

struct MergeParams {
  const float* part;
  const RunHead* head;
  const RunInfo* info;
  const int32_t* flags;
  uint16_t* o;
  int32_t* status;
  const unsigned long long* tree;
  float scale_log2;
  int Hq, Hkv, D, C, ctas, words;  // C: runs
};

constexpr int kMergeWarps = 16;
constexpr int kMergeThreads = 32 * kMergeWarps;
constexpr int kFewRows = 16, kFewStates = 4;
static_assert(kMaxCtas <= kMergeThreads, "a thread per run");

// Joins the partial states of the tiles that runs' borders cut. Every block
// finds out from the runs' heads which tiles those are, a run per thread, and
// takes its share of them, in items:
//   kByRow (calls of few rows per tile, whose states lie row by row): a row by the
//     whole block, the states dealt out to its warps, which join theirs first and
//     then one another's in shared memory (decode over a long context: few rows,
//     many states), or 16 rows, a warp each, where there are few states;
//   else (cut tiles of prompts: many rows, few states; 4 head dims of all rows side by
//     side): 32 rows, a lane each, a warp per 16th of the head dims, state by state.
// The first run of a tile left its state in its second slot (a tile that the run's
// end cuts), the others in their first. An item's chain is two trips to memory, the
// heads, then all else. (A trip takes 0.7 us here, and more where many blocks read
// the same lines: 3 blocks per SM that read all of the runs' places took a decode
// call of 26 us to 31. The second form for all calls: a token of 8 ragged sequences
// 63 us for 55; the first for all: a prompt of 4096 109 for 102.)
template <bool kByRow>
__global__ void __launch_bounds__(kMergeThreads, 1) paged_merge_kernel(const MergeParams p) {
  __shared__ __align__(16) float s_acc[kMergeWarps][256];
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ RunHead s_head[kMergeThreads + 1];
  __shared__ unsigned s_ends[kMergeWarps];  // of runs: the next is not of the same tile
  __shared__ int s_sum[kMergeWarps];
  __shared__ int s_items[kMergeThreads + 1], s_c1[kMergeThreads];  // items before a run's tile's, the tile's last run
  __shared__ int s_first;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int C = p.C, t = threadIdx.x, lane = t & 31, warp = t >> 5, blocks = C * p.ctas;
  int2 h = make_int2(-1, 0);
  if (t < C) h = __ldcg(reinterpret_cast<const int2*>(p.head + t));
  s_head[t + 1] = RunHead{h.x, h.y};
  if (t == 0) s_head[0] = RunHead{-1, 0}, s_first = kMergeThreads, s_items[0] = 0;
  if (blockIdx.x == 0) {
    // the call's status: the outcome of the lowest-numbered block that failed
    const int failed = t < blocks ? __ldcg(p.flags + t) : 0;
    __syncthreads();
    if (failed) atomicMin(&s_first, t);
    __syncthreads();
    if (t == s_first) *p.status = failed;
    if (t == 0 && s_first == kMergeThreads) *p.status = 0;
  }
  __syncthreads();
  // Run t is its tile's second if it starts inside the tile and run t - 1, which
  // has the unit before, does not, or does at the first unit; the runs after it that
  // start in the tile follow one another.
  const RunHead before = s_head[t], next = t + 1 < kMergeThreads ? s_head[t + 2] : RunHead{-1, 0};
  const bool second = (h.y & 2) != 0 && !((before.what & 2) != 0 && before.tile == h.x);
  const unsigned ends = __ballot_sync(0xffffffffu, !(next.what != 0 && next.tile == h.x));
  if (lane == 0) s_ends[warp] = ends;
  __syncthreads();
  int items = 0, c1 = t;
  if (second) {
    unsigned e = s_ends[warp] & (~0u << lane);
    int w = warp;
    while (e == 0u) e = s_ends[++w];  // (the last thread's next is none)
    c1 = 32 * w + __ffs(e) - 1;
    const int there = h.y >> 2;
    items = !kByRow ? (there + 31) / 32
            : there <= kFewRows && c1 - t + 2 > kFewStates ? there
                                                           : (there + kMergeWarps - 1) / kMergeWarps;
  }
  int sum = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) s_sum[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (w == warp) sum += total;
    total += s_sum[w];
  }
  s_items[t + 1] = sum;
  s_c1[t] = c1;
  __syncthreads();
  const int r = p.Hq / p.Hkv, D = p.D, rows = kRows * p.ctas;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int c = 0;  // the last run with s_items[c] <= item
#pragma unroll
    for (int o = kMergeThreads / 2; o > 0; o >>= 1)
      if (s_items[c + o] <= item) c += o;
    const int c0 = c - 1, states = s_c1[c] - c0 + 1, there = s_head[c + 1].what >> 2, part = item - s_items[c];
    const int4 i0 = __ldcg(reinterpret_cast<const int4*>(p.info + c));      // g, rt
    const int4 i1 = __ldcg(reinterpret_cast<const int4*>(p.info + c) + 1);  // lo, n, len
    const float* first = p.part + (size_t)(2 * c0 + 1) * slot_floats(D, rows);
    const float* rest = p.part + (size_t)(2 * c0) * slot_floats(D, rows);
    auto state = [&](int k) {  // of run c0 + k
      return k == 0 ? first : rest + (size_t)2 * k * slot_floats(D, rows);
    };
    auto output = [&](int row) -> uint16_t* {  // null: a query that sees nothing has its zeros already
      const int rho = i0.y * rows + row, tok = rho / r;
      return i1.z - i1.y + tok < 0 ? nullptr
                                   : p.o + ((size_t)(i1.x + tok) * p.Hq + (size_t)i0.x * r + rho - tok * r) * D;
    };
    auto inverse = [&](float L, int row) -> float {
      const int tok = (i0.y * rows + row) / r;
      return L != 0.f ? 1.f / L : inverse_of_none(p.tree, p.words, i1.x + tok, tok, i1.z - i1.y);
    };
    if (kByRow) {
      const bool shared = there <= kFewRows && states > kFewStates;
      const int row = shared ? part : part * kMergeWarps + warp, from = shared ? warp : 0, step = shared ? kMergeWarps : 1;
      if (row >= there) continue;  // (not where the block shares a row)
      const int wide = D > 128 ? 2 : 1;
      const bool on = 4 * lane < D;
      constexpr int kAhead = 5;  // states that are asked for at once
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      float M = kMinusBig, L = 0.f;  // (all lanes alike)
#pragma unroll 1
      for (int base = from; base < states; base += kAhead * step) {
        float4 x[kAhead][2];
        float m[kAhead], l[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int s = base + k * step;
          x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          m[k] = kMinusBig;
          l[k] = 0.f;
          if (s < states) {
            const float* o = state(s);
            const float4* v = reinterpret_cast<const float4*>(o + (size_t)row * D) + lane;
            if (on) x[k][0] = __ldcg(v);
            if (wide == 2) x[k][1] = __ldcg(v + 32);
            m[k] = __ldcg(o + (size_t)D * rows + row);
            l[k] = __ldcg(o + (size_t)(D + 1) * rows + row);
          }
        }
        const float old = M;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) M = fmaxf(M, m[k]);
        const float f = ex2((old - M) * p.scale_log2);
        L *= f;
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i].x *= f, acc[i].y *= f, acc[i].z *= f, acc[i].w *= f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float e = ex2((m[k] - M) * p.scale_log2);
          L = fmaf(e, l[k], L);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            acc[i].x = fmaf(e, x[k][i].x, acc[i].x), acc[i].y = fmaf(e, x[k][i].y, acc[i].y);
            acc[i].z = fmaf(e, x[k][i].z, acc[i].z), acc[i].w = fmaf(e, x[k][i].w, acc[i].w);
          }
        }
      }
      uint16_t* out = output(row);
      if (!shared) {
        const float inv = inverse(L, row);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (on && i < wide && out != nullptr)
            *reinterpret_cast<uint2*>(out + 4 * lane + 128 * i) =
                make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
        continue;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (on && i < wide) *reinterpret_cast<float4*>(&s_acc[warp][4 * lane + 128 * i]) = acc[i];
      if (lane == 0) s_m[warp] = M, s_l[warp] = L;
      __syncthreads();
      if (t < D && out != nullptr) {
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, s_m[w]);
        float l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
          const float e = ex2((s_m[w] - M) * p.scale_log2);
          l = fmaf(e, s_l[w], l);
          o = fmaf(e, s_acc[w][t], o);
        }
        out[t] = __bfloat16_as_ushort(__float2bfloat16_rn(o * inverse(l, row)));
      }
      __syncthreads();
    } else {
      const int row = 32 * part + lane, per = D / 64;  // chunks of 4 head dims of a warp: 1, 2 or 4
      if (row >= there) continue;                      // (nobody waits for anyone here)
      constexpr int kAhead = 4;
      float4 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      float M = kMinusBig, L = 0.f;
#pragma unroll 1
      for (int base = 0; base < states; base += kAhead) {
        float4 x[kAhead][4];
        float m[kAhead], l[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          m[k] = kMinusBig;
          l[k] = 0.f;
          const bool on = base + k < states;
          const float* o = state(on ? base + k : 0);
          if (on) {
            m[k] = __ldcg(o + (size_t)D * rows + row);
            l[k] = __ldcg(o + (size_t)(D + 1) * rows + row);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && i < per) x[k][i] = __ldcg(reinterpret_cast<const float4*>(o) + (size_t)(warp * per + i) * rows + row);
          }
        }
        const float old = M;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) M = fmaxf(M, m[k]);
        const float f = ex2((old - M) * p.scale_log2);
        L *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i].x *= f, acc[i].y *= f, acc[i].z *= f, acc[i].w *= f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float e = ex2((m[k] - M) * p.scale_log2);
          L = fmaf(e, l[k], L);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[i].x = fmaf(e, x[k][i].x, acc[i].x), acc[i].y = fmaf(e, x[k][i].y, acc[i].y);
            acc[i].z = fmaf(e, x[k][i].z, acc[i].z), acc[i].w = fmaf(e, x[k][i].w, acc[i].w);
          }
        }
      }
      uint16_t* out = output(row);
      const float inv = inverse(L, row);
      if (out != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < per)
            *reinterpret_cast<uint2*>(out + 4 * (warp * per + i)) =
                make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
      }
    }
  }
}

// ================================================================= host ===

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Blocks that share a tile.
int tile_blocks(const moe_paged_shape& s) {
  return s.D >= 128 && (long long)s.T * s.Hq > 128ll * s.B * s.Hkv ? 2 : 1;
}

// Whether find_small and find_tiles serve a call: their tables hold its sequences,
// its tiles are few enough and the places of all of them stay below 2^31.
bool narrow(const moe_paged_shape& s, int rows) {
  const long long tiles = (long long)s.T * (s.Hq / s.Hkv) / rows + s.B;
  const long long units = (long long)s.max_pages * s.page / kKeys + 2;
  return s.B <= kSmall && tiles <= kSmallTiles && tiles * s.Hkv * (units + kTileCost) <= 0x7FFFFFFFll;
}

size_t workspace_bytes(const moe_paged_shape& s) {
  // as many slots of 128 rows for pairs as for single blocks
  return 256 + kMaxCtas * (sizeof(int32_t) + sizeof(RunHead) + sizeof(RunInfo)) +
         2 * kMaxCtas * slot_floats(s.D, kRows) * sizeof(float);
}

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

// 4-D map of a pool [n_pages Hkv][page][D], the head dims as D / 64 slabs of 64
// outside the positions, with boxes of `rows` positions, or a page's where it has
// fewer, by `slabs` slabs (by one there, unless `whole`), in the 128-byte swizzle;
// pages past the pool read as zeros.
cudaError_t pool_map(CUtensorMap* m, const void* base, const moe_paged_shape& s, int rows, int slabs, bool whole) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {64, (cuuint64_t)s.page, (cuuint64_t)s.D / 64, (cuuint64_t)s.n_pages * s.Hkv};
  const cuuint64_t strides[3] = {(cuuint64_t)s.D * 2, 128, (cuuint64_t)s.page * s.D * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(rows < s.page ? rows : s.page),
                             (cuuint32_t)(whole || rows <= s.page ? slabs : 1), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

moe_status attn(const moe_paged_shape* shape, const void* q, const moe_paged_cache* cache, const int32_t* offsets,
                const int32_t* lens, const uint64_t* tree, float scale, void* o, void* workspace, size_t ws_bytes,
                void* stream, int stalled = -1, long long timeout_ns = kv8::kTimeoutNs) {
  if (!shape) return MOE_ERR_INVALID_ARG;
  const moe_paged_shape s = *shape;
  if (!shape_ok(s)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!cache_ok(cache) || !aligned(offsets, 4) || !aligned(lens, 4) || !aligned(q, 16) || !aligned(o, 16) ||
      !aligned(tree, 8) || !workspace || !aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  const float scale_log2 = scale * kLog2e;  // of all kernels of the call
  if (!(scale > 0.f) || !(scale_log2 < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < workspace_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.T == 0) {
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), st);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "status clear");
  }
  if (!q || !offsets || !lens || !o || (s.tree_words > 0) != (tree != nullptr)) return MOE_ERR_INVALID_ARG;
  const int sms = kv8::sm_count(), ctas = tile_blocks(s);
  if (sms <= 0) return cuda_fail(cudaErrorInvalidDevice, "device query");
  const int runs = (sms < kMaxCtas ? sms : kMaxCtas) / ctas;
  if (runs < 1) return cuda_fail(cudaErrorInvalidDevice, "multiprocessors");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  int32_t* flags = reinterpret_cast<int32_t*>(ws + 256);
  RunHead* head = reinterpret_cast<RunHead*>(flags + kMaxCtas);
  RunInfo* info = reinterpret_cast<RunInfo*>(head + kMaxCtas);
  float* part = reinterpret_cast<float*>(info + kMaxCtas);
  const int r = s.Hq / s.Hkv;
  const bool by_row = (long long)s.T * s.Hq <= kByRowRows * (long long)s.B * s.Hkv;
  const Params prm{static_cast<const uint16_t*>(q), offsets, lens, cache->tables,
                   reinterpret_cast<const unsigned long long*>(tree), static_cast<uint16_t*>(o), part, head, info, flags,
                   scale_log2, by_row ? 0.f : kSlack, s.B, s.T, s.Hq, s.Hkv, page_shift(s.page), s.n_pages, s.max_pages, s.tree_words,
                   s.q_stride ? s.q_stride : s.Hq * s.D, ((1ull << 36) + r - 1) / r,
                   (long long)s.T * s.Hq > 32ll * s.B * s.Hkv ? kTileCost : kFewRowsCost, by_row,
                   narrow(s, kRows * ctas), stalled, timeout_ns};
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
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const auto go = [&](auto d, auto n) -> cudaError_t {
    using F = Cfg<decltype(d)::value, decltype(n)::value>;
    const auto kernel = paged_attn_kernel<decltype(d)::value, decltype(n)::value>;
    static SmemLimitMemo smem_memo;
    CUtensorMap tk, tv;
    cudaError_t e = pool_map(&tk, cache->k_pages, s, F::kKeyRows, F::kSlabsK, false);
    if (e == cudaSuccess) e = pool_map(&tv, cache->v_pages, s, F::kKeysV, F::kSlabsV, true);
    if (e == cudaSuccess) e = ensure_smem(kernel, F::kBytes, &smem_memo);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = F::kBytes;
    return cudaLaunchKernelEx(&cfg, kernel, tk, tv, prm);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  cudaError_t e;
  if (s.D == 64) e = go(std::integral_constant<int, 64>{}, One{});
  else if (s.D == 128 && ctas == 1) e = go(std::integral_constant<int, 128>{}, One{});
  else if (s.D == 128) e = go(std::integral_constant<int, 128>{}, Two{});
  else if (ctas == 1) e = go(std::integral_constant<int, 256>{}, One{});
  else e = go(std::integral_constant<int, 256>{}, Two{});
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  const MergeParams mp{part, head, info, flags, static_cast<uint16_t*>(o), status, prm.tree,
                       scale_log2, s.Hq, s.Hkv, s.D, runs, ctas, s.tree_words};
  const long long most = by_row ? (long long)s.T * s.Hq : sms;  // no more items than rows
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  e = by_row ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<true>, mp)
             : cudaLaunchKernelEx(&cfg, paged_merge_kernel<false>, mp);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "paged merge launch");
}

}  // namespace
}  // namespace paged
}  // namespace bgmoe

extern "C" {

moe_status moe_paged_workspace_bytes(const moe_paged_shape* shape, size_t* bytes) {
  if (!shape || !bytes) return MOE_ERR_INVALID_ARG;
  if (!bgmoe::paged::shape_ok(*shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = bgmoe::paged::workspace_bytes(*shape);
  return MOE_OK;
}

moe_status moe_paged_attn(const moe_paged_shape* shape, const void* q, const moe_paged_cache* cache,
                          const int32_t* offsets, const int32_t* lens, const uint64_t* tree, float scale, void* o,
                          void* workspace, size_t ws_bytes, void* stream) {
  return bgmoe::paged::attn(shape, q, cache, offsets, lens, tree, scale, o, workspace, ws_bytes, stream);
}

moe_status moe_paged_attn_test_stall(const moe_paged_shape* shape, const void* q, const moe_paged_cache* cache,
                                     const int32_t* offsets, const int32_t* lens, const uint64_t* tree, float scale,
                                     void* o, void* workspace, size_t ws_bytes, int32_t stalled_block,
                                     int64_t timeout_ns, void* stream) {
  if (stalled_block < 0 || timeout_ns <= 0 || timeout_ns > bgmoe::kv8::kTimeoutNs) return MOE_ERR_INVALID_ARG;
  return bgmoe::paged::attn(shape, q, cache, offsets, lens, tree, scale, o, workspace, ws_bytes, stream, stalled_block,
                            timeout_ns);
}

}  // extern "C"
