// Device pieces that the attention kernels share: matrix products, LDS, loads straight to it.
#ifndef KDACONV_ATTENTION_DEVICE_H_
#define KDACONV_ATTENTION_DEVICE_H_

#include "latent_device.h"

namespace kdaconv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int kF>
__device__ __forceinline__ f32x4 mfma_16x16x32(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kF == kRuleBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
}

template <int kF>
__device__ __forceinline__ f32x16 mfma_32x32x16(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (kF == kRuleBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ u32x4 lds_read16(const lds_char* p) {
  return *(const __attribute__((address_space(3))) u32x4*)p;
}

// Of a group of 16 lanes, lane i gives the address of 4 elements, columns 4 (i % 4) .. of row
// i / 4, and gets column i of the 4 rows.
__device__ __forceinline__ u32x2 lds_read_columns(const lds_char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)const_cast<lds_char*>(p)));
}

// 16 bytes per lane from memory to LDS, at the wave's place + 16 times the lane's number. Not the
// builtin: the compiler would wait for all such loads before any LDS read that follows. Who
// reads the bytes waits for them (s_waitcnt vmcnt), and for the barrier if another wave loads.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: the compiler sets it before each use
__device__ __forceinline__ void to_lds16(const char* from, lds_char* wave_to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(from), "s"((uint32_t)(uintptr_t)wave_to) : "memory", "m0");
}
// The same at `offset` bytes from an address that all lanes share.
__device__ __forceinline__ void to_lds16(const char* base, uint32_t offset, lds_char* wave_to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(offset), "s"(base), "s"((uint32_t)(uintptr_t)wave_to) : "memory", "m0");
}

#pragma clang diagnostic pop

// A barrier for LDS alone: __syncthreads() would also wait for the loads under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Pairs of elements with 0 in the place of infinities and NaN.
template <int kF>
__device__ __forceinline__ u32x4 finite_pairs(u32x4 x) {
  constexpr uint32_t kHigh = kF == kRuleBF16 ? 0x7F800000u : 0x7C000000u, kLow = kHigh >> 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((x[i] & kHigh) == kHigh) x[i] &= 0xFFFFu;
    if ((x[i] & kLow) == kLow) x[i] &= 0xFFFF0000u;
  }
  return x;
}

// Hides that x is the same in every iteration of a loop. Without it the compiler works out
// all rows' offsets before the loop, and spills them.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Memory that a load need not take for LDS: waits for such flat loads are waits for all of them.
template <class X>
using Global = const __attribute__((address_space(1))) X*;

// What a key outside the sequence, and channels past a latent's, read.
static __device__ const uint32_t kZeros[kLatentMax / 2] = {};

// A row's largest score may grow by this (in powers of two) before its sums are rescaled.
constexpr float kSlack = 8.0f;
constexpr float kLowest = -3.402823466e38f;

}  // namespace kdaconv

#endif  // KDACONV_ATTENTION_DEVICE_H_
