// Expanded attention over packed sequences: parameters shared by the host code and the kernels.
#ifndef KDACONV_EXPANDED_ATTENTION_H_
#define KDACONV_EXPANDED_ATTENTION_H_

#include "latent.h"

namespace kdaconv {

constexpr int kExpandKeys = 64;  // keys per step
constexpr int kWaveRows = 32;  // queries per wave

struct ExpandParams {
  const char* q;
  const char* k;
  const char* kr;
  const char* v;
  char* out;  // (tokens, heads, value channels), contiguous
  const int32_t* qsl;
  const int32_t* ksl;
  int64_t q_ts, q_hs, k_ts, k_hs, kr_ts, v_ts, v_hs;  // bytes; kr_ts is k_ts if rope is 0
  int32_t tokens, keys, seqs, heads;
  int32_t dim, rope, vdim;
  int32_t programs;  // blocks of rows: sequence s owns v(s) = s + start of s / rows up to v(s + 1)
  int32_t search_top;  // 64^(levels - 1), 64^levels >= seqs
  float scale;  // times log2(e), positive; 1 if `vanish`
  bool vanish;  // the scale is 0, or too small for FP32
  uint32_t flip;  // the queries' sign bits, where the scale was negative
  bool causal;
  int32_t splits;  // parts of a block's keys, each a workgroup's
  float* partial;  // if there are several: per program, head and part an ExpandPartial
};

// A part's sums, then each row's exponent and weight.
struct ExpandPartial {
  int rows, channels;
  __host__ __device__ constexpr int64_t floats() const { return (int64_t)rows * (channels + 2); }
  __host__ __device__ constexpr int64_t exponent() const { return (int64_t)rows * channels; }
  __host__ __device__ constexpr int64_t weight() const { return (int64_t)rows * (channels + 1); }
};

template <int kF, int kDim, int kRope, int kWaves>
void launch_expanded(const ExpandParams& P, hipStream_t st);

}  // namespace kdaconv

#endif  // KDACONV_EXPANDED_ATTENTION_H_
