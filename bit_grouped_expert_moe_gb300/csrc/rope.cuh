// Norm and rotation of heads (include/rope.h), as moe_rope and the paged
// cache's append do them.
//
// A head of D values is D / 16 lanes' (a power of two of lanes, the last idle
// where D / 16 is none), two pieces of 8 values each: a rotating lane's pieces
// hold both halves of 8 pairs, pairs 8 l .. 8 l + 7 of lane l in either layout,
// so a pair never leaves its lane and one lane's angles serve both layouts.
// The norm is a sum over the head's lanes.
//
// Angles are turns in 64-bit fixed point: position times the table's entry,
// modulo 2^64, without a reduction of large angles and without a table of
// sines as long as the context. A lane computes its 8 once and uses them for
// all heads that it takes of the token.
#pragma once

#include "common.cuh"
#include "rope.h"

namespace bgmoe {
namespace rope {

// Host checks shared by the entry points (rope.cu).
bool spec_ok(const moe_rope_spec& s, int D);  // values
bool spec_pointers_ok(const moe_rope_spec& s);

struct Spec {
  const uint64_t* turns;
  const uint16_t* gain[2];  // q, k
  int rot, pairs, norm;
  float eps, offset, magnitude;
};
Spec device_spec(const moe_rope_spec* s);  // of NULL: neither norm nor rotation

// lanes of a head, as a power of two
__host__ __device__ constexpr int head_lanes(int D) {
  return D <= 16 ? 1 : D <= 32 ? 2 : D <= 64 ? 4 : D <= 128 ? 8 : 16;
}

// The two pieces of lane l, as offsets in the head; none past D.
struct Pieces {
  int a, b;
  bool on, turns;
  __device__ Pieces(int l, int D, const Spec& s) {
    on = 16 * l < D;
    turns = 16 * l < s.rot;
    const bool apart = turns && !s.pairs;
    a = apart ? 8 * l : 16 * l;
    b = apart ? 8 * l + s.rot / 2 : 16 * l + 8;
  }
};

// Cosines and sines of a lane's 8 pairs at a position.
struct Angles {
  float c[8], s[8];
  __device__ void at(const Spec& sp, int l, int position) {
    const uint4* t = reinterpret_cast<const uint4*>(sp.turns + 8 * l);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ld_once_v4(t + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = w[i / 2];
      const uint64_t turn = (i & 1) ? ((uint64_t)x.w << 32 | x.z) : ((uint64_t)x.y << 32 | x.x);
      const int32_t at = (int32_t)((turn * (uint64_t)(int64_t)position) >> 32);  // 2^-32 turns, -2^31 .. 2^31 - 1
      sincospif((float)at * 4.656612873077393e-10f, &s[i], &c[i]);               // in half turns
      s[i] *= sp.magnitude;
      c[i] *= sp.magnitude;
    }
  }
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One head's two pieces, normed (`norm`, by the whole group of kLanes lanes
// alike) and rotated. Every lane of the warp calls it: the sum over a head goes
// by shuffles.
template <int kLanes>
__device__ __forceinline__ void apply(const Spec& s, const Pieces& p, const Angles& ang, bool norm,
                                      const uint16_t* gain, int D, uint4& va, uint4& vb) {
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  if (__any_sync(0xffffffffu, norm)) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float f = rsqrtf(sum / (float)D + s.eps);
    // A finite head whose squares pass fp32: the same of 2^-72 times its values,
    // beside whose squares (2^-24 at least, 2^120 at most in all) eps is nothing.
    if (__any_sync(0xffffffffu, !(sum < 3e38f))) {
      const bool large = !(sum < 3e38f);
      const float d = large ? 2.117582368135751e-22f : 1.f;  // 2^-72
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= norm ? d : 1.f;
        b[i] *= norm ? d : 1.f;
        t = fmaf(a[i], a[i], fmaf(b[i], b[i], t));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (large) f = rsqrtf(t / (float)D);
    }
    if (norm) {
      float ga[8], gb[8];
      if (gain != nullptr && p.on) {
        unpack8(ld_once_v4(gain + p.a), ga);
        unpack8(ld_once_v4(gain + p.b), gb);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= gain != nullptr ? f * (s.offset + ga[i]) : f;
        b[i] *= gain != nullptr ? f * (s.offset + gb[i]) : f;
      }
    }
  }
  if (p.turns) {
    if (s.pairs) {
      // pieces a, b hold pairs 8 l .. + 3 and + 4 .. + 7, both values of a pair side by side
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
        a[2 * i] = x * ang.c[i] - y * ang.s[i];
        a[2 * i + 1] = y * ang.c[i] + x * ang.s[i];
        b[2 * i] = z * ang.c[i + 4] - w * ang.s[i + 4];
        b[2 * i + 1] = w * ang.c[i + 4] + z * ang.s[i + 4];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = a[i], y = b[i];
        a[i] = x * ang.c[i] - y * ang.s[i];
        b[i] = y * ang.c[i] + x * ang.s[i];
      }
    }
  }
  va = pack8(a);
  vb = pack8(b);
}

}  // namespace rope
}  // namespace bgmoe
