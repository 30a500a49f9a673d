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

}  // namespace kv8
}  // namespace bgmoe
