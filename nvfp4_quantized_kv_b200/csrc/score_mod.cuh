// score_mod.cuh -- the score modifications of the masked attention
// (nvkv_score_mod in include/nvkv.h): a tanh cap, a bias that falls with the
// distance, and the visible key interval of a query.
//
// The attention kernels are templates over a Mod type: NoMod is the plain
// causal attention (every member folds away), ScoreMod the masked one.
#pragma once

#include "nvkv_common.cuh"

namespace nvkv {

constexpr float kLog2e = 1.4426950408889634f;

// tanh(u) = u P(u^2) for |u| <= kCapSmall, off by at most 1.9e-7, and by 2.8e-6
// of its value (a degree-9 odd polynomial, least maximum error by reweighted
// least squares over the interval); increasing for every u.
__host__ __device__ constexpr float tanh_coefficient(int i) {
  return i == 0   ? 0.9999972283f
         : i == 1 ? -0.3332307647f
         : i == 2 ? 0.1322609151f
         : i == 3 ? -0.04928044419f
                  : 0.01231882928f;
}
constexpr float kCapSmall = 0.75f;
constexpr float kCapSmallTanh = 0.635148f;  // tanh(0.75), rounded down

// Visible keys [lo, hi) of a query at position p of a sequence of kv_len
// tokens: lo = max(0, start, p - W + 1), hi = p + 1, or p + min(P - p, W)
// when p lies inside the prefix P; at most kv_len.  W <= 0: no window.
// Always an interval; empty (hi <= lo) when p < 0, or when nothing from
// start on is below hi.
__host__ __device__ inline void key_range(int p, int kv_len, int start, int window, int prefix,
                                          int &lo, int &hi) {
  lo = start > 0 ? start : 0;
  hi = lo;
  if (p < 0) return;
  hi = p + 1;
  if (window > 0 && p - window + 1 > lo) lo = p - window + 1;
  if (prefix > p) {
    const int ahead = prefix - p;
    hi = (window > 0 && window < ahead) ? p + window : prefix;
  }
  if (hi > kv_len) hi = kv_len;
}

// First key that any of the T newest queries of a sequence can see, and the
// 128-token units that hold the keys from there on (the split plan's units).
__host__ __device__ inline void visible_units(int kv_len, int T, int start, int window, int &lo,
                                              int &first_unit, int &units) {
  lo = start > 0 ? start : 0;
  const int p0 = kv_len > T ? kv_len - T : 0;  // position of the first query
  if (window > 0 && p0 - window + 1 > lo) lo = p0 - window + 1;
  if (kv_len <= 0 || lo >= kv_len) {
    first_unit = units = 0;
    return;
  }
  first_unit = lo / kUnitTokens;
  units = (kv_len - 1) / kUnitTokens - first_unit + 1;
}

// Plain causal attention.
struct NoMod {
  static constexpr bool kOn = false, kCap = false, kBias = false;
  __device__ __forceinline__ int units(const int32_t *kv_lens, int b, int) const {
    return units_of_len(kv_lens[b]);
  }
};

// Kernel arguments of the masked attention.  Scores are in base-2 units
// (x = q.k * sm_scale * log2 e), and so are the cap and the slopes.
struct ScoreMod {
  static constexpr bool kOn = true, kCap = true, kBias = false;
  float cap2;             // cap * log2 e; 0 = no cap
  float inv_cap;          // 1 / cap2
  float cap_top;          // see cap_small
  float poly[5];          // tanh's coefficients times cap2^(-2i)
  int window;             // 0 = none
  const float *slopes;    // [Hq] or null
  const int32_t *prefix;  // [batch] or null
  const int32_t *starts;  // decode: [batch], prefill: [total_q]; or null

  __device__ __forceinline__ int start(int i) const { return starts ? starts[i] : 0; }
  __device__ __forceinline__ int prefix_of(int b) const { return prefix ? prefix[b] : 0; }
  __device__ __forceinline__ float slope2(int hq) const { return slopes ? slopes[hq] * kLog2e : 0.f; }
  __device__ __forceinline__ int units(const int32_t *kv_lens, int b, int T) const {
    int lo, first, n;
    visible_units(kv_lens[b], T, start(b), window, lo, first, n);
    return n;
  }
  // cap2 * tanh(u), u = x / cap2, of two scores, off by at most about 3e-6
  // times the result (2^-18) at any cap and any x: near 0 the polynomial,
  // beyond it 1 - 2 / (exp(2 u) + 1) from one base-2 exponential and one
  // reciprocal, whose error of some 2^-21 of a cap would be whole units of a
  // score at a cap of 1e6.  (tanh.approx would be off by 2^-11 of a cap,
  // several per cent of a softmax weight at a cap of 50.)  The exponential's
  // overflow to infinity gives +cap2, its underflow -cap2.
  __device__ __forceinline__ float2 cap(float2 x) const {
    const float2 u = mul_f32x2(x, make_float2(inv_cap, inv_cap));
    const float2 v = mul_f32x2(u, u);
    float2 p = make_float2(tanh_coefficient(4), tanh_coefficient(4));
#pragma unroll
    for (int i = 3; i >= 0; --i)
      p = fma_f32x2(p, v, make_float2(tanh_coefficient(i), tanh_coefficient(i)));
    p = mul_f32x2(p, u);
    auto far = [](float a) {
      float e, r;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * (2.f * kLog2e)));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
      return fmaf(-2.f, r, 1.f);
    };
    const float tx = fabsf(u.x) <= kCapSmall ? p.x : far(u.x);
    const float ty = fabsf(u.y) <= kCapSmall ? p.y : far(u.y);
    return mul_f32x2(make_float2(tx, ty), make_float2(cap2, cap2));
  }
};

// cap() of two scores x with |x| <= kCapSmall * cap2, x P((x / cap2)^2) with
// the powers of cap2 in the coefficients: 5 packed instructions a pair.  The
// result is increasing in x for every x, so one of at most cap_top =
// kCapSmallTanh * cap2 shows that x was in the interval.  Caps whose powers
// leave fp32 (cap2 outside [1e-4, 3e4]) have a cap_top of -1: no result
// passes.
__device__ __forceinline__ float2 cap_small(const ScoreMod &m, float2 x) {
  const float2 v = mul_f32x2(x, x);
  float2 p = make_float2(m.poly[4], m.poly[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) p = fma_f32x2(p, v, make_float2(m.poly[i], m.poly[i]));
  return mul_f32x2(p, x);
}

// A ScoreMod whose call is known to cap, or to bias, its scores or not to. The
// tensor-core kernels are instances of these: code that a call does not run
// still takes room in the instruction caches that the warp roles of an SM
// share (decode_qk4 without cap and bias: 7 % faster when neither's code is
// there).
template <bool Cap, bool Bias>
struct ScoreModOf : ScoreMod {
  static constexpr bool kCap = Cap, kBias = Bias;
};

// Calls f with the ScoreModOf that a call needs.
template <class F>
auto with_mod(const ScoreMod &m, F &&f) {
  auto as = [&](auto mod) {
    static_cast<ScoreMod &>(mod) = m;
    return f(mod);
  };
  if (m.cap2 > 0.f)
    return m.slopes ? as(ScoreModOf<true, true>{}) : as(ScoreModOf<true, false>{});
  return m.slopes ? as(ScoreModOf<false, true>{}) : as(ScoreModOf<false, false>{});
}

// A launch that, with `dependent`, may start while the kernel before it in the
// stream ends (programmatic dependent launch): the masked attention kernels and
// their merges wait for that kernel in the device code before they touch
// global memory, so the launches' latencies lie behind one another's work.
struct DependentLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  DependentLaunch(dim3 grid, int threads, int smem, cudaStream_t stream, bool dependent) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
  }
  DependentLaunch(const DependentLaunch &) = delete;  // cfg points into it
};

// Ranges that the split plan of U units really has: the masked attention deals
// them to at most U of the S splits, so that every range owns a unit and the
// merge meets no empty one; the plain plan has S.
template <class Mod>
__host__ __device__ __forceinline__ int64_t plan_ranges(int64_t U, int64_t S) {
  return Mod::kOn && U < S ? U : S;
}
__host__ __device__ __forceinline__ int64_t split_ranges(int64_t U, int64_t S) {
  return plan_ranges<ScoreMod>(U, S);
}
// range_begin and range_of_unit, with 32-bit divisions where the products fit
// (a 64-bit one is some 150 cycles of a small step's 10 microseconds).
__device__ __forceinline__ int64_t range_begin_mod(int64_t c, int64_t U, int64_t S) {
  const uint64_t n = (uint64_t)c * (uint64_t)U;
  return n >> 32 ? (int64_t)(n / (uint64_t)S) : (int64_t)((uint32_t)n / (uint32_t)S);
}
__device__ __forceinline__ int64_t range_of_unit_mod(int64_t u, int64_t U, int64_t S) {
  const uint64_t n = (uint64_t)(u + 1) * (uint64_t)S - 1;
  return (n | (uint64_t)U) >> 32 ? (int64_t)(n / (uint64_t)U)
                                 : (int64_t)((uint32_t)n / (uint32_t)U);
}

// locate_pair over the units that a Mod's queries can see (T: queries per
// sequence of the whole step).
template <class Mod>
__device__ __forceinline__ void locate_pair_mod(const Mod &mod, const int32_t *kv_lens, int B,
                                                int Hkv, int T, int64_t u, int &b, int &h,
                                                int64_t &pair_start, int &units) {
  int64_t acc = 0;
  for (b = 0; b < B; ++b) {
    const int ub = mod.units(kv_lens, b, T);
    const int64_t span = (int64_t)ub * Hkv;
    if (u < acc + span) {
      h = (int)((u - acc) / ub);
      pair_start = acc + (int64_t)h * ub;
      units = ub;
      return;
    }
    acc += span;
  }
  h = 0;
  pair_start = acc;
  units = 0;
}

template <class Mod>
__device__ __forceinline__ int64_t total_units(const Mod &mod, const int32_t *kv_lens, int B,
                                               int Hkv, int T) {
  int64_t U = 0;
  for (int b = 0; b < B; ++b) U += (int64_t)mod.units(kv_lens, b, T) * Hkv;
  return U;
}

// First token of unit u of a pair that owns units [pair_start, pair_start +
// units).  With a distance bias a pair's units go from the newest to the
// oldest: the largest scores come first, so the running maximum is found once
// instead of being raised in every tile.  (Without one the ascending order is
// 2 % faster.)
template <class Mod>
__device__ __forceinline__ int unit_token(int first_unit, int units, int64_t pair_start,
                                          int64_t u) {
  const int i = (int)(u - pair_start);
  return (Mod::kBias ? first_unit + units - 1 - i : first_unit + i) * kUnitTokens;
}

}  // namespace nvkv
