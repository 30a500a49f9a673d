// Host-side launchers of the 8-bit cache's attention kernels.
#pragma once

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
};

// Split-context kernels (kv8_split.cu), for few query tokens per sequence.
size_t split_workspace_bytes(const moe_kv8_shape& s);
moe_status launch_split(const AttnArgs& a, cudaStream_t stream);

// Tensor-core tile kernels (kv8_tiles.cu), for many.
size_t tiles_workspace_bytes(const moe_kv8_shape& s);
moe_status launch_tiles(const AttnArgs& a, cudaStream_t stream);

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
  __device__ bool empty(int c) const { return per == 0 && c >= more; }
  __device__ int of(long long s) const {  // the run that holds place s
    const long long lead = more * (per + 1);
    return s < lead ? (int)div_small(s, per + 1) : more + (int)div_small(s - lead, per);
  }
};

}  // namespace kv8
}  // namespace bgmoe
