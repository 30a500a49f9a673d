// Norm and rotation of heads (include/rope.h), as moe_rope and the paged
// cache's append do them.
//
// A head of D values is D / 16 lanes' (a power of two of lanes, the last idle
// where D / 16 is none), two pieces of 8 values each, so that the first pieces
// of neighbouring lanes lie side by side, as do the second (whole sectors per
// load), and a pair never leaves its lane: with halves, a rotating lane's pieces
// are the two halves of 8 pairs. The norm is a sum over the head's lanes.
//
// Angles are turns in 64-bit fixed point: position times the table's entry,
// modulo 2^64, without a reduction of large angles and without a table of
// sines as long as the context. A warp computes those of its tokens once, a few
// per lane, into shared memory, for all heads that it takes.
//
// Bound: a call of few heads by one chain (table and values, angles, the stores:
// 64 tokens of 16 and 2 heads of 256 2.7 us in a graph, appended to pages 3.2);
// one of many by HBM (8192 tokens of 40 and 8 heads of 128 34 us, 6.0 TB/s of the
// 6.8 that a copy reaches): a head is read once and written once.
#pragma once

#include "common.cuh"
#include "rope.h"

namespace bgmoe {
namespace rope {

// Host checks shared by the entry points (rope.cu).
bool spec_ok(const moe_rope_spec& s, int D);  // values
bool spec_pointers_ok(const moe_rope_spec& s);

struct Spec {
  const unsigned long long* turns;
  const uint16_t* gain[2];  // q, k
  int rot, pairs, norm;
  float eps, offset, magnitude;
};
Spec device_spec(const moe_rope_spec* s);  // of NULL: neither norm nor rotation

// lanes of a head, as a power of two
__host__ __device__ constexpr int head_lanes(int D) {
  return D <= 16 ? 1 : D <= 32 ? 2 : D <= 64 ? 4 : D <= 128 ? 8 : 16;
}

// The two pieces of lane l, as offsets in the head, and their first pairs; none past D.
struct Pieces {
  int a, b, pair_a, pair_b;
  bool on, turn_a, turn_b;
  __device__ Pieces(int l, int D, const Spec& s) {
    const int lanes = D / 16, turning = s.rot / 16;
    on = l < lanes;
    if (s.pairs) {  // every piece holds 4 whole pairs
      a = 8 * l;
      b = 8 * (l + lanes);
      turn_a = on && a < s.rot;
      turn_b = on && b < s.rot;
      pair_a = a / 2;
      pair_b = b / 2;
    } else {
      const bool turns = l < turning;
      a = turns ? 8 * l : 8 * (l + turning);
      b = turns ? 8 * (l + turning) : 8 * (l + lanes);
      turn_a = turn_b = turns;
      pair_a = 8 * l;
      pair_b = 8 * l + 4;
    }
  }
};

// Cosine and sine of a pair at a position, times the magnitude.
__device__ __forceinline__ float2 angle(const Spec& s, uint64_t turns, int position) {
  const int32_t at = (int32_t)((turns * (uint64_t)(int64_t)position) >> 32);  // 2^-32 turns, -2^31 .. 2^31 - 1
  float2 v;
  sincospif((float)at * 4.656612873077393e-10f, &v.y, &v.x);  // in half turns
  return make_float2(v.x * s.magnitude, v.y * s.magnitude);
}

// Two fp32 values at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 w, x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 w, {%6, %7};\n"
      " fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The factor first: a value over the root mean square is sqrt(D) at most, while the
// factor times a gain may pass fp32, or fall below it.
__device__ __forceinline__ void scale8(float2 (&x)[4], const float* gain, float f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 g = *reinterpret_cast<const float4*>(gain + 4 * i);
    x[2 * i] = mul2(mul2(x[2 * i], make_float2(f, f)), make_float2(g.x, g.y));
    x[2 * i + 1] = mul2(mul2(x[2 * i + 1], make_float2(f, f)), make_float2(g.z, g.w));
  }
}
// 4 pairs side by side.
__device__ __forceinline__ void turn4(float2 (&x)[4], const float* cosines, const float* sines) {
  const float4 c = *reinterpret_cast<const float4*>(cosines), s = *reinterpret_cast<const float4*>(sines);
  const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = fma2(x[i], make_float2(cs[i], cs[i]), mul2(make_float2(x[i].y, x[i].x), make_float2(-sn[i], sn[i])));
}

// One head's two pieces, normed (`norm`, by the whole group of kLanes lanes
// alike) and rotated. Every lane of the warp calls it: the sum over a head goes
// by shuffles. cosines, sines: of the token's first pair; gain: of the head's
// first value.
template <int kLanes>
__device__ __forceinline__ void apply(const Spec& s, const Pieces& p, const float* cosines, const float* sines, bool norm,
                                      const float* gain, float inv_D, uint4& va, uint4& vb) {
  float2 a[4], b[4];
  unpack8(va, a);
  unpack8(vb, b);
  if (__any_sync(0xffffffffu, norm)) {
    float2 two = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) two = fma2(a[i], a[i], fma2(b[i], b[i], two));
    float sum = two.x + two.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float mean = fmaf(sum, inv_D, s.eps);
    float f = rsqrtf(mean);
    // A finite head whose squares pass fp32, or whose mean with eps does: the same of
    // 2^-72 times its values and 2^-144 times eps.
    if (__any_sync(0xffffffffu, !(mean < 3e38f))) {
      constexpr float kDown = 2.117582368135751e-22f;  // 2^-72
      const bool large = !(mean < 3e38f);
      const float d = large && norm ? kDown : 1.f;
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = mul2(a[i], make_float2(d, d));
        b[i] = mul2(b[i], make_float2(d, d));
        t = fmaf(a[i].x, a[i].x, fmaf(a[i].y, a[i].y, fmaf(b[i].x, b[i].x, fmaf(b[i].y, b[i].y, t))));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (large) f = rsqrtf(fmaf(t, inv_D, s.eps * kDown * kDown));
    }
    if (norm && p.on) {
      scale8(a, gain + p.a, f);
      scale8(b, gain + p.b, f);
    }
  }
  if (s.pairs) {
    if (p.turn_a) turn4(a, cosines + p.pair_a, sines + p.pair_a);
    if (p.turn_b) turn4(b, cosines + p.pair_b, sines + p.pair_b);
  } else if (p.turn_a) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float4 c = *reinterpret_cast<const float4*>(cosines + p.pair_a + 2 * i);
      const float4 n = *reinterpret_cast<const float4*>(sines + p.pair_a + 2 * i);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 cs = k == 0 ? make_float2(c.x, c.y) : make_float2(c.z, c.w);
        const float2 sn = k == 0 ? make_float2(n.x, n.y) : make_float2(n.z, n.w);
        const float2 x = a[i + k], y = b[i + k];
        a[i + k] = fma2(x, cs, mul2(y, make_float2(-sn.x, -sn.y)));
        b[i + k] = fma2(y, cs, mul2(x, sn));
      }
    }
  }
  va = pack8(a);
  vb = pack8(b);
}

// ------------------------------------------------------------- the pass ---

constexpr int kThreads = 128;
constexpr int kMaxTokens = 32;   // of a warp
constexpr int kMaxAngles = 512;

// What a warp takes: `tokens` tokens, `heads` of their H heads.
struct Split {
  int T, H, D, tokens, heads, chunks;  // chunks of the heads
};

// A call's warps: as many heads each as it has slots while the call's heads
// leave the GPU's warps idle (latency), then `ahead` times as many.
inline Split split(int T, int H, int D, int rot, int ahead, long long* blocks) {
  const int slots = 32 / head_lanes(D);
  const int room = (long long)T * H <= 152ll * 16 * slots ? slots : slots * ahead;  // heads of a warp
  Split s{T, H, D, 1, H, 1};
  if (H > room) {
    s.chunks = (H + room - 1) / room;
    s.heads = (H + s.chunks - 1) / s.chunks;
    s.heads = (s.heads + slots - 1) / slots * slots;
    s.chunks = (H + s.heads - 1) / s.heads;
  } else {
    s.tokens = room / H;
    if (s.tokens > kMaxTokens) s.tokens = kMaxTokens;
    if (rot > 0 && s.tokens > kMaxAngles / (rot / 2)) s.tokens = kMaxAngles / (rot / 2);
  }
  const long long warps = (long long)((T + s.tokens - 1) / s.tokens) * s.chunks;
  *blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return s;
}

// Io gives the heads their places:
//   Token                          what a block keeps of a token
//   bool token(t, &k, &position)   looks it up; false: nothing of it is written
//   kind(h)                        0 query, 1 key, 2 left as it is
//   from(t, h), to(k, t, h)        where head h lies and goes
//   refuse()                       a token was not to be written
// A slot is the lanes of one head. It asks for its kAhead heads (a warp has no
// more than kAhead times its slots) before the warp
// looks up its tokens and computes their angles. Warps do not wait for one
// another, so one's loads run beside another's sines: with blocks that shared
// their angles, 4096 tokens of 16 and 2 heads of 256 took 23 us for 19.
template <int kLanes, int kAhead, class Io>
__device__ __forceinline__ void turn(const Io& io, const Spec& sp, const Split& sl) {
  constexpr int kSlots = 32 / kLanes;
  struct Shared {
    float cosine[kMaxAngles], sine[kMaxAngles];
    typename Io::Token token[kMaxTokens];
    int position[kMaxTokens];
    bool ok[kMaxTokens];
  };
  __shared__ __align__(16) Shared shared[kThreads / 32];
  __shared__ __align__(16) float s_gain[2][256];
  const int lane = threadIdx.x & 31, l = lane % kLanes, slot = lane / kLanes;
  Shared& sh = shared[threadIdx.x >> 5];
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long group = w / sl.chunks;
  const int h0 = (int)(w - group * sl.chunks) * sl.heads;
  // a warp past the call's end has nothing to do but to help with the gains
  const int t0 = (int)min(group * sl.tokens, (long long)sl.T);
  const int nt = min(sl.tokens, sl.T - t0), nh = min(sl.heads, sl.H - h0), units = nt * nh;
  const Pieces pc(l, sl.D, sp);
  const float inv_D = 1.f / (float)sl.D;
  // unit u is head u % nh of token u / nh; a step of kSlots units in both
  const int step_t = kSlots / nh, step_h = kSlots - step_t * nh;
  uint4 a[kAhead], b[kAhead];
  {
    int t = slot / nh, h = slot - t * nh;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i * kSlots + slot < units && pc.on) {
        const uint16_t* x = io.from(t0 + t, h0 + h);
        a[i] = ld_once_v4(x + pc.a);
        b[i] = ld_once_v4(x + pc.b);
      }
      t += step_t;
      h += step_h;
      if (h >= nh) {
        h -= nh;
        ++t;
      }
    }
  }
  const int per = sp.rot / 2;
  const unsigned long long first = lane < per ? ld(sp.turns + lane) : 0;
  if (lane < nt) {
    int position = 0;
    const bool ok = io.token(t0 + lane, &sh.token[lane], &position);
    if (!ok) io.refuse();
    sh.ok[lane] = ok;
    sh.position[lane] = position;
  }
  if (sp.norm != 0) {
    for (int d = threadIdx.x; d < 2 * sl.D; d += kThreads) {
      const int k = d >= sl.D, e = k ? d - sl.D : d;
      const uint16_t* g = k ? sp.gain[1] : sp.gain[0];
      s_gain[k][e] = g != nullptr ? sp.offset + bf16_bits_to_f32(ld(g + e)) : 1.f;
    }
    __syncthreads();
  }
  __syncwarp();
  for (int i = lane, t = 0, j = lane; i < nt * per; i += 32) {
    while (j >= per) {
      j -= per;
      ++t;
    }
    const float2 v = angle(sp, i < min(per, 32) ? first : ld(sp.turns + j), sh.position[t]);
    sh.cosine[i] = v.x;
    sh.sine[i] = v.y;
    j += 32;
  }
  __syncwarp();
  int t = slot / nh, h = slot - t * nh;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (i * kSlots >= units) break;  // the whole warp alike
    const bool live = i * kSlots + slot < units;
    const int tok = live ? t : 0, kind = io.kind(h0 + h);
    uint4 x = a[i], y = b[i];
    apply<kLanes>(sp, pc, sh.cosine + tok * per, sh.sine + tok * per, kind < 2 && (sp.norm >> kind) & 1,
                  s_gain[kind & 1], inv_D, x, y);
    if (kind == 2) {
      x = a[i];
      y = b[i];
    }
    if (live && pc.on && sh.ok[tok]) {
      uint16_t* to = io.to(sh.token[tok], t0 + tok, h0 + h);
      *reinterpret_cast<uint4*>(to + pc.a) = x;
      *reinterpret_cast<uint4*>(to + pc.b) = y;
    }
    t += step_t;
    h += step_h;
    if (h >= nh) {
      h -= nh;
      ++t;
    }
  }
}

}  // namespace rope
}  // namespace bgmoe
