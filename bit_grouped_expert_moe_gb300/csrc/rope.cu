// Rotary positions (include/rope.h): the table of turns (host) and the pass
// that norms and rotates queries and keys.
//
// rope.cuh has the pass itself.
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "rope.cuh"

namespace bgmoe {
namespace rope {

bool spec_ok(const moe_rope_spec& s, int D) {
  if (s.rot < 0 || s.rot % 16 != 0 || s.rot > D) return false;
  if (s.layout != MOE_ROPE_HALF && s.layout != MOE_ROPE_PAIRS) return false;
  if (s.norm & ~(MOE_ROPE_NORM_Q | MOE_ROPE_NORM_K)) return false;
  // (with 1e-30 beside the mean square, squares that fall below fp32 miss nothing)
  return std::isfinite(s.eps) && (s.norm == 0 || s.eps >= 1e-30f) && std::isfinite(s.gain_offset) &&
         std::isfinite(s.magnitude);
}

bool spec_pointers_ok(const moe_rope_spec& s) {
  const auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return (s.rot == 0 || s.turns != nullptr) && a16(s.turns) && a16(s.q_gain) && a16(s.k_gain);
}

Spec device_spec(const moe_rope_spec* s) {
  if (s == nullptr) return Spec{};
  return Spec{reinterpret_cast<const unsigned long long*>(s->turns),
              {static_cast<const uint16_t*>(s->q_gain), static_cast<const uint16_t*>(s->k_gain)},
              s->rot,
              s->layout == MOE_ROPE_PAIRS, s->norm, s->eps, s->gain_offset, s->magnitude};
}

namespace {

// Heads in flight per slot, and blocks per SM (registers). us for 8192 tokens of 40
// and 8 heads of 128, and for 4096 of 16 and 2 of 256: 4, 4 41 and 23; 4, 5 38 and 20;
// 4, 6 35 and 19; 3, 6 37 and 18; 3, 7 37 and 17; 2, 8 40 and 19.
constexpr int kAhead = 4, kBlocks = 6;

struct Io {
  const uint16_t* x[2];  // q, k
  uint16_t* y[2];
  long long xs[2], ys[2];  // elements from token to token
  const int32_t* positions;
  int Hq, D;
  struct Token {};
  __device__ bool token(int t, Token*, int* position) const {
    if (positions != nullptr) *position = ld(positions + t);
    return true;
  }
  __device__ int kind(int h) const { return h >= Hq; }
  __device__ const uint16_t* from(int t, int h) const {
    return h < Hq ? x[0] + t * xs[0] + (long long)h * D : x[1] + t * xs[1] + (long long)(h - Hq) * D;
  }
  __device__ uint16_t* to(const Token&, int t, int h) const {
    return h < Hq ? y[0] + t * ys[0] + (long long)h * D : y[1] + t * ys[1] + (long long)(h - Hq) * D;
  }
  __device__ void refuse() const {}
};

template <int kLanes>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const Io io, const Spec spec, const Split split) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  turn<kLanes, kAhead>(io, spec, split);
}

bool shape_ok(const moe_rope_shape& s) {
  if (s.T < 0 || s.T > (1 << 24) || s.Hq < 0 || s.Hq > 4096 || s.Hk < 0 || s.Hk > 4096 || s.Hq + s.Hk == 0) return false;
  if ((long long)s.T * (s.Hq + s.Hk) > (1 << 30)) return false;
  if (s.D < 16 || s.D > 256 || s.D % 16 != 0) return false;
  const auto stride_ok = [](int v, long long least) { return v == 0 || (v % 8 == 0 && v >= least); };
  const long long q = (long long)s.Hq * s.D, k = (long long)s.Hk * s.D;
  return stride_ok(s.q_stride, q) && stride_ok(s.k_stride, k) && stride_ok(s.qo_stride, q) && stride_ok(s.ko_stride, k);
}

}  // namespace
}  // namespace rope
}  // namespace bgmoe

extern "C" {

moe_status moe_rope_table(const moe_rope_frequencies* f, uint64_t* turns, float* magnitude) {
  if (!f || !turns || !magnitude) return MOE_ERR_INVALID_ARG;
  if (f->rot < 16 || f->rot > 256 || f->rot % 16 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (f->scaling < MOE_ROPE_PLAIN || f->scaling > MOE_ROPE_RAMP || f->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (!(f->base > 1.0) || !std::isfinite(f->base) || !(f->factor >= 1.0) || !std::isfinite(f->factor))
    return MOE_ERR_INVALID_ARG;
  const bool by_turns = f->scaling == MOE_ROPE_BANDS || f->scaling == MOE_ROPE_RAMP;
  if (by_turns && (f->original < 1 || !(f->low > 0.0) || !(f->high > f->low) || !std::isfinite(f->high)))
    return MOE_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const auto index_of = [&](double t) { return f->rot * std::log(f->original / (two_pi * t)) / (2.0 * std::log(f->base)); };
  double lo = 0.0, hi = 1.0;
  if (f->scaling == MOE_ROPE_RAMP) {
    lo = std::fmax(std::floor(index_of(f->high)), 0.0);
    hi = std::fmin(std::ceil(index_of(f->low)), (double)f->rot - 1.0);
  }
  if (f->given != nullptr)
    for (int i = 0; i < f->rot / 2; ++i)
      if (!std::isfinite(f->given[i])) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < f->rot / 2; ++i) {
    double w = f->given != nullptr ? f->given[i] : std::pow(f->base, -2.0 * i / f->rot);
    const double stretched = w / f->factor;
    if (f->scaling == MOE_ROPE_LINEAR) {
      w = stretched;
    } else if (f->scaling == MOE_ROPE_BANDS) {
      const double t = f->original * std::fabs(w) / two_pi;
      const double keep = std::fmin(std::fmax((t - f->low) / (f->high - f->low), 0.0), 1.0);
      w = w * keep + stretched * (1.0 - keep);
    } else if (f->scaling == MOE_ROPE_RAMP) {
      const double u = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w * (1.0 - u) + stretched * u;
    }
    double turn = w / two_pi;
    turn -= std::floor(turn);  // 0 .. 1: a whole turn per position is none
    const double scaled = std::ldexp(turn, 64);
    turns[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
  }
  *magnitude = f->scaling == MOE_ROPE_RAMP ? (float)(0.1 * std::log(f->factor) + 1.0) : 1.f;
  return MOE_OK;
}

moe_status moe_rope(const moe_rope_shape* shape, const moe_rope_spec* spec, const void* q, const void* k,
                    const int32_t* positions, void* q_out, void* k_out, void* stream) {
  using namespace bgmoe;
  using namespace bgmoe::rope;
  if (!shape || !spec) return MOE_ERR_INVALID_ARG;
  const moe_rope_shape s = *shape;
  if (!shape_ok(s) || !spec_ok(*spec, s.D)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const auto bad = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; };
  if (bad(q, 16) || bad(k, 16) || bad(q_out, 16) || bad(k_out, 16) || bad(positions, 4) || !spec_pointers_ok(*spec))
    return MOE_ERR_INVALID_ARG;
  if (s.T == 0) return MOE_OK;
  if ((s.Hq > 0 && (!q || !q_out)) || (s.Hk > 0 && (!k || !k_out)) || (spec->rot > 0 && !positions))
    return MOE_ERR_INVALID_ARG;
  const Io io{{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k)},
              {static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(k_out)},
              {s.q_stride ? s.q_stride : (long long)s.Hq * s.D, s.k_stride ? s.k_stride : (long long)s.Hk * s.D},
              {s.qo_stride ? s.qo_stride : (long long)s.Hq * s.D, s.ko_stride ? s.ko_stride : (long long)s.Hk * s.D},
              spec->rot > 0 ? positions : nullptr, s.Hq, s.D};
  long long blocks = 0;
  const Split sl = split(s.T, s.Hq + s.Hk, s.D, spec->rot, kAhead, &blocks);
  const int lanes = head_lanes(s.D);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto go = [&](auto n) {
    return cudaLaunchKernelEx(&cfg, rope_kernel<decltype(n)::value>, io, device_spec(spec), sl);
  };
  const cudaError_t e = lanes == 1   ? go(std::integral_constant<int, 1>{})
                        : lanes == 2 ? go(std::integral_constant<int, 2>{})
                        : lanes == 4 ? go(std::integral_constant<int, 4>{})
                        : lanes == 8 ? go(std::integral_constant<int, 8>{})
                                     : go(std::integral_constant<int, 16>{});
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "rotation launch");
}

}  // extern "C"
