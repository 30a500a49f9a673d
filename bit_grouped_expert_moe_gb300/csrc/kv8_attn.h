// Host-side launchers of the 8-bit cache's attention kernels.
#pragma once

#include <atomic>

#include "kv8.cuh"

namespace bgmoe {
namespace kv8 {

struct AttnArgs {
  const uint16_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* offsets;
  const int32_t* lens;
  uint16_t* o;
  void* workspace;
  int B, T, Hq, Hkv, D, L_max, nblk, block, e4m3, q_stride;
  float scale_log2;  // scale * log2(e)
  int stalled;       // grid block that never brings its operands (tests), or -1
  long long timeout_ns;  // limit of every wait
};

constexpr long long kTimeoutNs = 1000000000ll;

// Split-context kernels (kv8_split.cu), for few query tokens per sequence.
size_t split_workspace_bytes(const moe_kv8_shape& s);
void split_steps(const moe_kv8_shape& s, long long* T);  // the most tokens with 8, and with 16 rows per tile
moe_status launch_split(const AttnArgs& a, cudaStream_t stream);

// Tensor-core tile kernels (kv8_tiles.cu), for many.
size_t tiles_workspace_bytes(const moe_kv8_shape& s);
moe_status launch_tiles(const AttnArgs& a, cudaStream_t stream);

// V scales far apart. With x = score + log2 s_v, a row's sum L = sum w / s_v comes
// from weights w = 2^(x - m + 7), which are zero below 2^-126. Let S be the
// largest V scale that the tile's units have shown so far: L is 2^7 / S at least,
// and a position whose weight was lost had less than 2^-126 / s_v in it. Where
// s_v >= kFar S that is less than 2^-45 of L, and there is no more to do. Positions
// below (blocks of zeros have the smallest scale) are summed without the detour,
// as 2^(x - m + 7 - log2 s_v), and kLift times that, so that what is lost of them
// is less than 2^-158 against 2^7 / 2^121, 2^-44 of L. (x <= m + 8 and s_v >= 2^-60
// keep it below 2^108.) For the same reason L goes from one m to another in two
// steps, by the square root of the factor: the factor itself may be below 2^-126.
constexpr float kFar = 3.2311742677852644e-27f;       // 2^-88
constexpr float kLiftBits = 32.f, kUnlift = 2.3283064365386963e-10f;  // 2^-32

int sm_count();  // of the current device, or 0 (kv8_attn.cu)

// How the work is laid out, by both kinds: the rows of a (sequence, KV head)
// are its r = Hq / Hkv query heads of every query token, token by token; row
// tiles are RT consecutive rows; a tile's units are the runs of KT positions
// that its last row sees: none, when a sequence has more queries than
// positions.
__device__ __forceinline__ int seq_tiles(int n, int r, int RT) { return (n * r + RT - 1) / RT; }
__device__ __forceinline__ int tile_units(int n, int len, int r, int RT, int KT, int rt) {
  const int last = min(n * r, (rt + 1) * RT) - 1;
  const int see = len - n + last / r + 1;
  return see > 0 ? (see + KT - 1) / KT : 0;
}

// sum_{i < n} floor((a i + b) / m) for a, b >= 0, by the Euclidean recursion
// on (m, a): whole parts of a / m and b / m are summed directly, and what is
// left counts lattice points under a line, which are counted along the other
// axis.
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (true) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) return sum;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
}

// Units of the tiles before tile k of a sequence. A whole tile's
// ceil((len - n + floor(last / r) + 1) / KT), with last = RT (rt + 1) - 1, is
// floor((RT rt + c) / (r KT)) with c = RT - 1 + r (len - n + KT), a line in rt.
__device__ inline long long units_before(int n, int len, int r, int RT, int KT, int k) {
  const int all = seq_tiles(n, r, RT);
  long long sum = 0;
  if (k <= 4) {
    for (int rt = 0; rt < k; ++rt) sum += tile_units(n, len, r, RT, KT, rt);
    return sum;
  }
  if (k == all) sum += tile_units(n, len, r, RT, KT, --k);  // the last tile may be ragged
  const long long c = RT - 1 + (long long)r * ((long long)len - n + KT);
  const long long k0 = c < 0 ? (-c + RT - 1) / RT : 0;      // tiles before see nothing
  if (k0 < k) sum += floor_sum(k - k0, (long long)r * KT, RT, c + RT * k0);
  return sum;
}

// Tiles at the start of a sequence whose rows see no position.
__device__ __forceinline__ int empty_tiles(int n, int len, int r, int RT) {
  if (n <= len) return 0;
  const int all = seq_tiles(n, r, RT);  // the last row sees len positions
  return len == 0 ? all : min(all - 1, (r * (n - len) + RT) / RT - 1);
}

// N places dealt out to C grid blocks in contiguous runs, the first N % C of
// them one place longer. 64-bit divisions cost hundreds of cycles, and there is
// no work of another kind to hide them behind, so small numbers are divided in
// 32 bits.
__device__ __forceinline__ long long div_small(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
struct Runs {
  long long per;  // N / C
  int more;       // N % C
  __device__ Runs(long long N, int C) : per(div_small(N, C)), more((int)(N - per * C)) {}
  __device__ long long start(int c) const { return c * per + min(c, more); }
};

// Runs are cut on a scale of places, where a tile with units takes `cost` more
// places than units, before its first: what beginning and ending a tile costs
// a run.
__device__ inline long long places_before(int n, int len, int r, int RT, int KT, int cost, int k) {
  return units_before(n, len, r, RT, KT, k) + (long long)cost * max(k - empty_tiles(n, len, r, RT), 0);
}

// The first unit at or after a place: unit i of the nb of row tile rt of KV head
// g of sequence b (b = -1: past the last), which owns tokens lo .. lo + n - 1 and
// len positions; the units before it, and its tile's number in the order
// (sequence, KV head, row tile).
struct Place {
  int b, g, rt, i, nb, tile, lo, n, len;
  long long units;
};

// By one warp: checks the tables (false if they break the rules), counts the
// call's places and finds that of run c's start.
__device__ inline bool find_run(const int32_t* offsets, const int32_t* lens, int B, int T, int Hkv, int L_max, int r,
                                int RT, int KT, int cost, int c, int C, Place* out) {
  const int lane = threadIdx.x & 31;
  long long total = 0, before = 0, units = 0, at = 0;
  int tiles = 0;
  bool bad = false;
  Place k{};
  k.b = -1;
  // Pass 0 counts, pass 1 searches: one copy of the code, which runs cold.
#pragma unroll 1
  for (int base = 0, pass = 0; base < B;) {
    const int b = base + lane;
    long long v1 = 0, w1 = 0;  // this lane's sequence, per KV head: places, units
    int nt1 = 0, lo = 0, hi = 0, len = 0;
    if (b < B) {
      lo = ld(offsets + b), hi = ld(offsets + b + 1), len = ld(lens + b);
      if (offsets_bad(lo, hi, b, B, T) || len < 0 || len > L_max) {
        bad = true;
      } else {
        nt1 = seq_tiles(hi - lo, r, RT);
        w1 = units_before(hi - lo, len, r, RT, KT, nt1);
        v1 = w1 + (long long)cost * (nt1 - empty_tiles(hi - lo, len, r, RT));
      }
    }
    const long long v = v1 * Hkv, w = w1 * Hkv;
    const int nt = nt1 * Hkv;
    long long vi = v, wi = w;
    int ti = nt;
#pragma unroll 1
    for (int o = 1; o < min(B, 32); o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, vi, o), y = __shfl_up_sync(0xffffffffu, wi, o);
      const int z = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) {
        vi += x;
        wi += y;
        ti += z;
      }
    }
    const int end = min(B, 32) - 1;  // the last lane that the sums reach
    const long long all = __shfl_sync(0xffffffffu, vi, end);
    base += 32;
    if (pass == 0) {
      total += all;
      if (base < B) continue;
      bad = __any_sync(0xffffffffu, bad);
      if (bad) break;
      at = Runs(total, C).start(c);
      pass = 1;
      if (B > 32) {  // else the search goes on with this chunk
        base = 0;
        continue;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + vi > at);
    if (hit) {
      const int L = __ffs(hit) - 1;
      k.b = base - 32 + L;
      long long off = at - (before + __shfl_sync(0xffffffffu, vi - v, L));
      const long long per = __shfl_sync(0xffffffffu, v1, L), per_units = __shfl_sync(0xffffffffu, w1, L);
      units += __shfl_sync(0xffffffffu, wi - w, L);
      tiles += __shfl_sync(0xffffffffu, ti - nt, L);
      k.lo = __shfl_sync(0xffffffffu, lo, L);
      k.n = __shfl_sync(0xffffffffu, hi, L) - k.lo;
      k.len = __shfl_sync(0xffffffffu, len, L);
      const int all_tiles = __shfl_sync(0xffffffffu, nt1, L);
      k.g = (int)div_small(off, per);
      off -= k.g * per;
      // the last tile whose first place is at or before off, 32 candidates a
      // round (tiles without units share their successor's first place: the
      // search ends on the last of them, which has some)
      int a = 0, z = all_tiles;
#pragma unroll 1
      while (z - a > 1) {
        const int step = (z - a + 31) / 32, cand = a + lane * step;
        const bool in = cand < z && places_before(k.n, k.len, r, RT, KT, cost, cand) <= off;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));
        a += last * step;
        z = min(z, a + step);
      }
      k.rt = a;
      k.nb = tile_units(k.n, k.len, r, RT, KT, a);
      const long long first = units_before(k.n, k.len, r, RT, KT, a);
      k.i = max((int)(off - first) - cost * (max(a - empty_tiles(k.n, k.len, r, RT), 0) + 1), 0);
      units += k.g * per_units + first + k.i;
      k.tile = tiles + k.g * all_tiles + a;
      break;
    }
    before += all;
    units += __shfl_sync(0xffffffffu, wi, end);
    tiles += __shfl_sync(0xffffffffu, ti, end);
  }
  k.units = units;
  *out = k;
  return !bad;
}

// Moves registers between a block's warpgroups: every warp of a group calls one
// of the two. A share above a thread's registers at launch waits until the
// other groups have given theirs, so the shares add up to what the block was
// launched with, which launch_registers checks before the first launch.
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <class Kernel>
cudaError_t launch_registers(Kernel kernel, int regs, std::atomic<bool>* known) {
  if (known->load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return e;
  if (a.numRegs != regs) return cudaErrorInvalidKernelImage;
  known->store(true, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace kv8
}  // namespace bgmoe
