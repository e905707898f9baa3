// Device pieces of the latent attention kernels: vectors of elements, angles, 8-bit codes.
#ifndef KDACONV_LATENT_DEVICE_H_
#define KDACONV_LATENT_DEVICE_H_

#include "delta_rule_device.h"
#include "latent.h"

namespace kdaconv {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // aligned to elements only

// 8 neighbouring elements in FP32, at any multiple of their size.
template <int kF>
__device__ __forceinline__ void load_eight(const char* p, float (&v)[8]) {
  if constexpr (kF == kRuleF32) {
    const f32x4 a = ((const f32x4a4*)p)[0], b = ((const f32x4a4*)p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const u32x4 r = *(const u32x4_any*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = Pair<kF>::value(r[i]);
      v[2 * i] = a.x;
      v[2 * i + 1] = a.y;
    }
  }
}

template <int kF>
__device__ __forceinline__ u32x4 pack_eight(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 a = {v[2 * i], v[2 * i + 1]};
    if constexpr (kF == kRuleBF16)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
    else
      r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, f16x2));
  }
  return r;
}

template <int kF>
__device__ __forceinline__ void store_eight(char* p, const float (&v)[8]) {
  if constexpr (kF == kRuleF32) {
    ((f32x4a4*)p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    ((f32x4a4*)p)[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *(u32x4_any*)p = pack_eight<kF>(v);
  }
}

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, bool wide) {
  return wide ? ((const int64_t*)p)[i] : (int64_t)((const int32_t*)p)[i];
}

// Cosine and sine of position * frequency, for positions up to 2^53. The product is taken in FP64 with
// its rounding's error beside it (0 up to positions of 2^29), and counted in turns, with 1 / (2 pi)
// in two parts. What is left, at most half a turn, rounds to FP32: off by 2^-26 of a turn at
// most, however far the position.
__device__ __forceinline__ f32x2 turn(int64_t position, float frequency) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double a = (double)position * (double)frequency;
  const double low = __builtin_fma((double)position, (double)frequency, -a);
  const double turns = a * kHi;
  const double rest = __builtin_fma(low, kHi, __builtin_fma(a, kLo, __builtin_fma(a, kHi, -turns)));
  const double left = (turns - __builtin_rint(turns)) + rest;
  // (Turns from 2^50 on are counted in quarters, and the rest is up to an eighth.)
  const float t = (float)(left - __builtin_rint(left));
  float s, c;
  sincospif(2.0f * t, &s, &c);
  return f32x2{c, s};
}

// (u, v) turned; each product and sum rounded in FP32.
__device__ __forceinline__ f32x2 turned(float u, float v, f32x2 cs) {
  return f32x2{__builtin_fmaf(u, cs.x, -(v * cs.y)), __builtin_fmaf(u, cs.y, v * cs.x)};
}

// The scale byte of a block whose largest finite magnitude is `most`: the smallest exponent e,
// at least -100, with most <= 448 * 2^e, plus 127. 448 is 1.75 * 2^8.
__device__ __forceinline__ int scale_byte(float most) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, most);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  return (e < -100 ? -100 : e) + 127;
}

// 2^(byte - 127), for bytes 1 to 254; 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// Two e4m3 codes, the lower or upper half of a word, times a scale: what scale_value(byte) times
// the code's value is when rounded once to 16 bits, for all codes and bytes.
template <int kF, bool kHigh>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t codes, float scale) {
  if constexpr (kF == kRuleBF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, kHigh));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, kHigh));
}

}  // namespace kdaconv

#endif  // KDACONV_LATENT_DEVICE_H_
