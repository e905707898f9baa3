// Device pieces that the kernels of the gated delta rule share: element access, the gate,
// sequence metadata and sums over lanes.
#ifndef KDACONV_DELTA_RULE_DEVICE_H_
#define KDACONV_DELTA_RULE_DEVICE_H_

#include "delta_rule.h"

namespace kdaconv {

// Formats (the interface's codes).
constexpr int kRuleBF16 = KDACONV_BF16;
constexpr int kRuleF16 = KDACONV_F16;
constexpr int kRuleF32 = KDACONV_F32;

constexpr float kLog2e = 1.44269504088896340736f;
// exp(-104) is below half the smallest FP32 subnormal: a log decay under it is a full
// reset, and clamping it there keeps running sums of resets (and of -infinity) finite.
constexpr float kMinLogDecay = -104.0f;

// Vectors of elements. They need only be aligned to their elements: the memory pipeline
// takes vectors at any such address, and a Q|K|V slice may start at any column.
typedef uint32_t u32a2 __attribute__((aligned(2)));
typedef uint32_t u32a4 __attribute__((aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x2 f32x2a4 __attribute__((aligned(4)));
typedef f32x4 f32x4a4 __attribute__((aligned(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int kF>
constexpr int elem_bytes() {
  return kF == kRuleF32 ? 4 : 2;
}

// A pair of neighbouring elements as loaded, and its two values.
template <int kF>
struct Pair {
  typedef uint32_t raw;
  static __device__ __forceinline__ raw load(const char* p) { return *(const u32a2*)p; }
  static __device__ __forceinline__ f32x2 value(raw r) {
    if constexpr (kF == kRuleBF16) {
      return f32x2{__builtin_bit_cast(float, r << 16), __builtin_bit_cast(float, r & 0xFFFF0000u)};
    } else {
      const f16x2 h = __builtin_bit_cast(f16x2, r);
      return f32x2{(float)h.x, (float)h.y};
    }
  }
  static __device__ __forceinline__ void store(char* p, f32x2 v) {
    if constexpr (kF == kRuleBF16)
      *(u32a2*)p = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    else
      *(u32a2*)p = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
  static __device__ __forceinline__ raw zero() { return 0u; }
};

template <>
struct Pair<kRuleF32> {
  typedef f32x2 raw;
  static __device__ __forceinline__ raw load(const char* p) { return *(const f32x2a4*)p; }
  static __device__ __forceinline__ f32x2 value(raw r) { return r; }
  static __device__ __forceinline__ void store(char* p, f32x2 v) { *(f32x2a4*)p = v; }
  static __device__ __forceinline__ raw zero() { return f32x2{0.0f, 0.0f}; }
};

template <int kF>
__device__ __forceinline__ float load_elem(const char* p) {
  if constexpr (kF == kRuleF32) return *(const float*)p;
  if constexpr (kF == kRuleF16) return (float)*(const _Float16*)p;
  return __builtin_bit_cast(float, (uint32_t)(*(const uint16_t*)p) << 16);
}

template <int kF>
__device__ __forceinline__ void store_elem(char* p, float v) {
  if constexpr (kF == kRuleF32)
    *(float*)p = v;
  else if constexpr (kF == kRuleF16)
    *(_Float16*)p = (_Float16)v;
  else
    *(__bf16*)p = (__bf16)v;
}

__device__ __forceinline__ bool is_finite(float x) { return __builtin_fabsf(x) < __builtin_huge_valf(); }
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigmoid_f(float x) {
  return rcp_hw(1.0f + exp2_hw(-kLog2e * x));
}

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1]. log1p(e) = 2 atanh(z)
// with z = e / (2 + e) <= 1/3: the odd series up to z^15, whose first term left out is
// below 2^-27 of the sum. Small results keep their relative precision, which the decay of
// slow channels lives on (an absolute error of 2^-24 in a log decay of 2^-10 would be a
// relative error of 2^-14 in the state such a channel gathers).
__device__ __forceinline__ float softplus_f(float x) {
  const float e = exp2_hw(-kLog2e * __builtin_fabsf(x));
  const float z = e * rcp_hw(2.0f + e);
  const float w = z * z;
  float p = 1.0f / 15.0f;
  p = __builtin_fmaf(p, w, 1.0f / 13.0f);
  p = __builtin_fmaf(p, w, 1.0f / 11.0f);
  p = __builtin_fmaf(p, w, 1.0f / 9.0f);
  p = __builtin_fmaf(p, w, 1.0f / 7.0f);
  p = __builtin_fmaf(p, w, 1.0f / 5.0f);
  p = __builtin_fmaf(p, w, 1.0f / 3.0f);
  p = __builtin_fmaf(p, w, 1.0f);
  return __builtin_fmaf(2.0f * z, p, __builtin_fmaxf(x, 0.0f));
}

// The gate of one head: log2 of the decay of a channel.
struct Gate {
  int mode;
  float a;  // -log2e * exp(a_log), or for the bounded gate log2e * exp(a_log)
  float lower;  // log2e * lower_bound
  bool deep;  // the bounded gate may reach kMinLogDecay

  __device__ __forceinline__ Gate(const RuleParams& P, int h) : mode(P.gate), a(0.0f) {
    if (mode != KDACONV_GATE_LOG) a = kLog2e * __builtin_expf(P.a_log[h]);
    if (mode == KDACONV_GATE_SOFTPLUS) a = -a;
    lower = kLog2e * P.lower_bound;
    deep = P.lower_bound < kMinLogDecay;
  }

  static __device__ __forceinline__ float clamp(float d) {
    return d < kLog2e * kMinLogDecay ? kLog2e * kMinLogDecay : d;  // a NaN stays one
  }

  __device__ __forceinline__ float soft(float g, float bias) const {
    return clamp(a * softplus_f(g + bias));
  }

  // shift: -a * bias
  __device__ __forceinline__ float bounded(float g, float shift) const {
    return lower * rcp_hw(1.0f + exp2_hw(__builtin_fmaf(-a, g, shift)));
  }

  // N pairs at once: one (uniform) branch on the kind of gate.
  template <int N>
  __device__ __forceinline__ void eval(f32x2 (&g)[N], f32x2 bias) const {
    if (mode == KDACONV_GATE_LOG) {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = f32x2{clamp(kLog2e * g[i].x), clamp(kLog2e * g[i].y)};
    } else if (mode == KDACONV_GATE_SOFTPLUS) {
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = f32x2{soft(g[i].x, bias.x), soft(g[i].y, bias.y)};
    } else {
      const f32x2 shift = {-a * bias.x, -a * bias.y};
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = f32x2{bounded(g[i].x, shift.x), bounded(g[i].y, shift.y)};
      if (deep) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = f32x2{clamp(g[i].x), clamp(g[i].y)};
      }
    }
  }
};

// A wave-uniform value, for the compiler.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The rows of sequence s, and where its state lives. Values out of range give an empty
// sequence or no line, never an access outside the arrays.
struct Sequence {
  int start, len;
  int64_t line;  // -1: no stored state
  bool init;  // starts from the line

  __device__ __forceinline__ Sequence(const RuleParams& P, int s) {
    if (P.qsl != nullptr) {
      int a = P.qsl[s], b = P.qsl[s + 1];
      a = a < 0 ? 0 : (a > P.num_tokens ? P.num_tokens : a);
      b = b < a ? a : (b > P.num_tokens ? P.num_tokens : b);
      start = a;
      len = b - a;
    } else {
      start = s;
      len = 1;
    }
    line = P.cache_indices[(int64_t)s * P.ci_stride];
    if (line < 0 || line >= P.num_cache_lines || (P.has_null_block && line == P.null_block_id))
      line = -1;
    init = line >= 0 && (P.all_init || (P.has_init != nullptr && P.has_init[s] != 0));
  }
};

__device__ __forceinline__ float beta_value(const RuleParams& P, int kF, int64_t token, int h) {
  const int64_t i = token * P.b_ts + h * P.b_hs;
  float b;
  if (P.beta_f32 || kF == kRuleF32)
    b = load_elem<kRuleF32>(P.beta + 4 * i);
  else if (kF == kRuleF16)
    b = load_elem<kRuleF16>(P.beta + 2 * i);
  else
    b = load_elem<kRuleBF16>(P.beta + 2 * i);
  return P.beta_logits ? sigmoid_f(b) : b;
}

// 1 / sqrt(x) as the sum of two FP32 values (0 for 0), by Newton's steps in FP64. Keys
// are scaled with both (k hi + k lo, rounded once): the rule applies I - beta k k^T once
// per token, so an error of 2^-24 in the length of equal keys, with no decay and beta
// near 2, would grow with every token (measured on 97 equal keys: 1.3e-5 of the largest
// output; 1e-6 with the pair).
struct Factor {
  float hi, lo;
};

__device__ __forceinline__ double inverse_root_f64(double x) {
  if (x == 0.0) return 0.0;
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(0.5 * y, __builtin_fma(-x * y, y, 1.0), y);
  return y;
}

__device__ __forceinline__ Factor two_floats(double y) {
  Factor f;
  f.hi = (float)y;
  f.lo = (float)(y - (double)f.hi);
  return f;
}

__device__ __forceinline__ Factor inverse_root(double x) { return two_floats(inverse_root_f64(x)); }

__device__ __forceinline__ float scaled(float x, Factor f) {
  return __builtin_fmaf(x, f.hi, x * f.lo);
}

template <int kWidth, class T>
__device__ __forceinline__ T lane_sum(T x) {
#pragma unroll
  for (int m = kWidth / 2; m > 0; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

}  // namespace kdaconv

#endif  // KDACONV_DELTA_RULE_DEVICE_H_
