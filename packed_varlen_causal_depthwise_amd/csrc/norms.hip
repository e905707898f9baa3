// The norms around the gated delta rule (include/kdaconv.h states both).
//
// Both are streams: every input is read once and every output written once, 16 bytes (8
// elements of the 16-bit formats) per lane and access, with a row held in registers
// between the sum of squares and the scaling. What bounds them is HBM.
//
// Inputs, and the residual on its way back, pass the caches by (non-temporal accesses): a
// call of some size reads its inputs once, and what it writes to the residual is read again
// only after the block between. That leaves the caches to the outputs, which the next
// product reads at once. With all accesses ordinary 16384 x 4096 bf16 residual rows took
// 98 us and 16384 tokens of 12 gated heads 32.9 us, against 82 (6.5 TB/s) and 30.2; with
// non-temporal outputs too 91 and 28.8. The gate's kind is a template argument: a branch per
// element on it kept the vector units busy for 73% of those 30.2 us, without it 26.2 (5.8
// TB/s).
#include "delta_rule_device.h"

#include <algorithm>

namespace kdaconv {
namespace {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef u32x4v u32x4a2 __attribute__((aligned(2)));

// 8 neighbouring elements as FP32.
struct Eight {
  float v[8];
};

// kOnce: the elements are not used again soon.
template <int kF, bool kOnce = false>
__device__ __forceinline__ Eight load8(const char* p) {
  Eight e;
  if constexpr (kF == kRuleF32) {
    const f32x4a4* const at = (const f32x4a4*)p;
    const f32x4 a = kOnce ? __builtin_nontemporal_load(at) : *at;
    const f32x4 b = kOnce ? __builtin_nontemporal_load(at + 1) : at[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e.v[i] = a[i];
      e.v[4 + i] = b[i];
    }
  } else {
    const u32x4a2* const at = (const u32x4a2*)p;
    const u32x4v r = kOnce ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = Pair<kF>::value(r[i]);
      e.v[2 * i] = a.x;
      e.v[2 * i + 1] = a.y;
    }
  }
  return e;
}

template <int kF, bool kOnce = false>
__device__ __forceinline__ void store8(char* p, const Eight& e) {
  if constexpr (kF == kRuleF32) {
    const f32x4 a = {e.v[0], e.v[1], e.v[2], e.v[3]}, b = {e.v[4], e.v[5], e.v[6], e.v[7]};
    f32x4a4* const at = (f32x4a4*)p;
    if constexpr (kOnce) {
      __builtin_nontemporal_store(a, at);
      __builtin_nontemporal_store(b, at + 1);
    } else {
      at[0] = a;
      at[1] = b;
    }
  } else {
    u32x4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = {e.v[2 * i], e.v[2 * i + 1]};
      if constexpr (kF == kRuleBF16)
        r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
      else
        r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, f16x2));
    }
    if constexpr (kOnce)
      __builtin_nontemporal_store(r, (u32x4a2*)p);
    else
      *(u32x4a2*)p = r;
  }
}

// The last elements of a row whose length is no multiple of 8.
template <int kF>
__device__ __forceinline__ Eight load_tail(const char* p, int n) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 8; ++i) e.v[i] = i < n ? load_elem<kF>(p + i * elem_bytes<kF>()) : 0.0f;
  return e;
}

template <int kF>
__device__ __forceinline__ void store_tail(char* p, const Eight& e, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store_elem<kF>(p + i * elem_bytes<kF>(), e.v[i]);
}

__device__ __forceinline__ float rsqrt_f(float x) { return 1.0f / __builtin_sqrtf(x); }

struct GatedNormParams {
  const char* x;
  const char* gate;
  const float* weight;
  char* out;
  int64_t x_s0, x_s1, g_s0, g_s1;
  int64_t rows;
  uint32_t heads, heads_magic;  // n / heads = (umulhi(n, magic) + n) >> shift
  int32_t heads_shift;
  int32_t dim;
  int32_t lanes_log;  // log2 of the lanes per row (a power of two >= dim / 8)
  float inv_dim, eps;
};

// kU rows per lane group: their loads are all issued before the first sum. Rows past the last
// load the last one and lanes past dim the row's start, so that no load waits for a branch.
template <int kF, int kU, int kGate>
__global__ __launch_bounds__(256) void gated_rms_norm_kernel(const GatedNormParams P) {
  constexpr int kEB = elem_bytes<kF>();
  const int lanes = 1 << P.lanes_log;
  const int c = 8 * (threadIdx.x & (lanes - 1));
  const int64_t groups = 256 >> P.lanes_log;
  const int64_t first = (int64_t)blockIdx.x * groups * kU + (threadIdx.x >> P.lanes_log);
  const bool in = c < P.dim;
  const int at = in ? c : 0;
  Eight x[kU], z[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t row = first + u * groups;
    const uint32_t n = (uint32_t)(row < P.rows ? row : P.rows - 1);
    const uint32_t t = (__umulhi(n, P.heads_magic) + n) >> P.heads_shift, h = n - t * P.heads;
    x[u] = load8<kF, true>(P.x + ((int64_t)t * P.x_s0 + (int64_t)h * P.x_s1 + at) * kEB);
    if constexpr (kGate != KDACONV_NORM_GATE_NONE)
      z[u] = load8<kF, true>(P.gate + ((int64_t)t * P.g_s0 + (int64_t)h * P.g_s1 + at) * kEB);
  }
  Eight w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w.v[i] = 1.0f;
  if (P.weight != nullptr) w = load8<kRuleF32>((const char*)(P.weight + at));
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t row = first + u * groups;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[u].v[i], x[u].v[i], s);
    s = in ? s : 0.0f;
    for (int m = lanes >> 1; m > 0; m >>= 1) s += __shfl_xor(s, m);
    const float r = rsqrt_f(__builtin_fmaf(s, P.inv_dim, P.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y = x[u].v[i] * r * w.v[i];
      if constexpr (kGate != KDACONV_NORM_GATE_NONE) y *= sigmoid_f(z[u].v[i]);
      if constexpr (kGate == KDACONV_NORM_GATE_SILU) y *= z[u].v[i];
      x[u].v[i] = y;
    }
    if (in && row < P.rows) store8<kF>(P.out + (row * P.dim + c) * kEB, x[u]);
  }
}

struct ResidualNormParams {
  const char* x;
  char* residual;
  const float* weight;
  char* out;
  int64_t x_stride, r_stride;
  int32_t hidden;
  float scale, inv_hidden, eps;
};

// One row per workgroup of kThreads, kV vectors of 8 per lane.
template <int kF, int kThreads, int kV>
__global__ __launch_bounds__(kThreads) void residual_rms_norm_kernel(const ResidualNormParams P) {
  constexpr int kEB = elem_bytes<kF>();
  const int64_t row = blockIdx.x;
  const char* const x = P.x + row * P.x_stride * kEB;
  char* const residual = P.residual == nullptr ? nullptr : P.residual + row * P.r_stride * kEB;
  Eight a[kV], b[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = 8 * (threadIdx.x + i * kThreads), n = P.hidden - c;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[i].v[e] = b[i].v[e] = 0.0f;
    if (n >= 8) {
      a[i] = load8<kF, true>(x + c * kEB);
      if (residual != nullptr) b[i] = load8<kF, true>(residual + c * kEB);
    } else if (n > 0) {
      a[i] = load_tail<kF>(x + c * kEB, n);
      if (residual != nullptr) b[i] = load_tail<kF>(residual + c * kEB, n);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = 8 * (threadIdx.x + i * kThreads), n = P.hidden - c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[i].v[e] = __builtin_fmaf(P.scale, a[i].v[e], b[i].v[e]);
      s = __builtin_fmaf(a[i].v[e], a[i].v[e], s);
    }
    if (residual != nullptr) {
      if (n >= 8)
        store8<kF, true>(residual + c * kEB, a[i]);
      else if (n > 0)
        store_tail<kF>(residual + c * kEB, a[i], n);
    }
  }
  s = lane_sum<kRuleWave>(s);
  if constexpr (kThreads > kRuleWave) {
    __shared__ float part[kThreads / kRuleWave];
    if (threadIdx.x % kRuleWave == 0) part[threadIdx.x / kRuleWave] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / kRuleWave; ++w) s += part[w];
  }
  const float r = rsqrt_f(__builtin_fmaf(s, P.inv_hidden, P.eps));
  char* const out = P.out + row * P.hidden * kEB;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = 8 * (threadIdx.x + i * kThreads), n = P.hidden - c;
    if (n <= 0) continue;
    if (P.weight != nullptr) {
      const Eight w = n >= 8 ? load8<kRuleF32>((const char*)(P.weight + c))
                             : load_tail<kRuleF32>((const char*)(P.weight + c), n);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i].v[e] *= r * w.v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i].v[e] *= r;
    }
    if (n >= 8)
      store8<kF>(out + c * kEB, a[i]);
    else
      store_tail<kF>(out + c * kEB, a[i], n);
  }
}

bool element_aligned(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == KDACONV_F32 ? 4 : 2) == 0;
}

bool known(int dtype) { return dtype == KDACONV_BF16 || dtype == KDACONV_F16 || dtype == KDACONV_F32; }

// Multiplier and shift of n / d for n < 2^31 (d >= 1): magic = ceil(2^(32 + L) / d) - 2^32
// with 2^L >= d.
void divider(uint32_t d, uint32_t* magic, int32_t* shift) {
  int l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  const unsigned __int128 num = (unsigned __int128)1 << (32 + l);
  *magic = (uint32_t)((num + d - 1) / d - ((unsigned __int128)1 << 32));
  *shift = l;
}

template <int kF, int kGate>
void launch_gated_as(const GatedNormParams& P, hipStream_t st) {
  const int64_t groups = 256 >> P.lanes_log;
  // Four rows per lane group where that still leaves every CU several workgroups; else one,
  // for latency.
  const int rows = P.rows >= groups * 4 * 1024 ? 4 : 1;
  const dim3 grid((unsigned)((P.rows + rows * groups - 1) / (rows * groups)));
  if (rows == 4)
    hipLaunchKernelGGL((gated_rms_norm_kernel<kF, 4, kGate>), grid, dim3(256), 0, st, P);
  else
    hipLaunchKernelGGL((gated_rms_norm_kernel<kF, 1, kGate>), grid, dim3(256), 0, st, P);
}

template <int kF>
void launch_gated(const GatedNormParams& P, int gate, hipStream_t st) {
  if (gate == KDACONV_NORM_GATE_SIGMOID)
    launch_gated_as<kF, KDACONV_NORM_GATE_SIGMOID>(P, st);
  else if (gate == KDACONV_NORM_GATE_SILU)
    launch_gated_as<kF, KDACONV_NORM_GATE_SILU>(P, st);
  else
    launch_gated_as<kF, KDACONV_NORM_GATE_NONE>(P, st);
}

template <int kF>
void launch_residual(const ResidualNormParams& P, int64_t rows, hipStream_t st) {
  const dim3 grid((unsigned)rows);
#define KDACONV_RESIDUAL(T, V) \
  hipLaunchKernelGGL((residual_rms_norm_kernel<kF, T, V>), grid, dim3(T), 0, st, P)
  if (P.hidden <= 512)
    KDACONV_RESIDUAL(64, 1);
  else if (P.hidden <= 1024)
    KDACONV_RESIDUAL(64, 2);
  else if (P.hidden <= 2048)
    KDACONV_RESIDUAL(256, 1);
  else if (P.hidden <= 4096)
    KDACONV_RESIDUAL(256, 2);
  else if (P.hidden <= 8192)
    KDACONV_RESIDUAL(256, 4);
  else
    KDACONV_RESIDUAL(256, 8);
#undef KDACONV_RESIDUAL
}

}  // namespace
}  // namespace kdaconv

using namespace kdaconv;

extern "C" int kdaconv_gated_rms_norm(const void* x, int dtype, int64_t num_tokens,
                                      int64_t num_heads, int64_t dim, int64_t x_stride0,
                                      int64_t x_stride1, const void* gate, int64_t gate_stride0,
                                      int64_t gate_stride1, int activation, const float* weight,
                                      double eps, void* out, kdaconv_stream_t stream) {
  if (num_tokens < 0 || num_heads < 0 || dim <= 0 || !known(dtype)) return KDACONV_EINVAL;
  if (activation != KDACONV_NORM_GATE_NONE && activation != KDACONV_NORM_GATE_SIGMOID &&
      activation != KDACONV_NORM_GATE_SILU)
    return KDACONV_EINVAL;
  if (!(eps >= 0.0)) return KDACONV_EINVAL;
  if (dim % 8 != 0 || dim > 512) return KDACONV_EUNSUPPORTED;
  if (x_stride0 < 0 || x_stride1 < 0 || gate_stride0 < 0 || gate_stride1 < 0)
    return KDACONV_EUNSUPPORTED;
  // A launch may not reach 2^32 threads; a workgroup of 256 takes 16 rows at least.
  constexpr int64_t kMaxRows = ((int64_t)1 << 28) - 16;
  if (num_tokens > kMaxRows || num_heads > kMaxRows || num_tokens * num_heads > kMaxRows)
    return KDACONV_EUNSUPPORTED;
  if (num_tokens == 0 || num_heads == 0) return KDACONV_OK;
  const bool gated = activation != KDACONV_NORM_GATE_NONE;
  if (!x || !out || (gated && !gate)) return KDACONV_EINVAL;
  if (!element_aligned(x, dtype) || !element_aligned(out, dtype) ||
      (gated && !element_aligned(gate, dtype)) || !element_aligned(weight, KDACONV_F32))
    return KDACONV_EUNSUPPORTED;
  GatedNormParams P;
  P.x = static_cast<const char*>(x);
  P.gate = static_cast<const char*>(gate);
  P.weight = weight;
  P.out = static_cast<char*>(out);
  P.x_s0 = x_stride0;
  P.x_s1 = x_stride1;
  P.g_s0 = gate_stride0;
  P.g_s1 = gate_stride1;
  P.rows = num_tokens * num_heads;
  P.heads = (uint32_t)num_heads;
  divider(P.heads, &P.heads_magic, &P.heads_shift);
  P.dim = (int32_t)dim;
  P.lanes_log = 0;
  while ((8 << P.lanes_log) < dim) ++P.lanes_log;
  P.inv_dim = (float)(1.0 / (double)dim);
  P.eps = (float)eps;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == KDACONV_F32)
    launch_gated<kRuleF32>(P, activation, st);
  else if (dtype == KDACONV_F16)
    launch_gated<kRuleF16>(P, activation, st);
  else
    launch_gated<kRuleBF16>(P, activation, st);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}

extern "C" int kdaconv_residual_rms_norm(const void* x, int dtype, int64_t num_tokens,
                                         int64_t hidden, int64_t x_stride, void* residual,
                                         int64_t residual_stride, double residual_scale,
                                         const float* weight, double eps, void* out,
                                         kdaconv_stream_t stream) {
  if (num_tokens < 0 || hidden <= 0 || !known(dtype)) return KDACONV_EINVAL;
  if (!(eps >= 0.0)) return KDACONV_EINVAL;
  if (hidden > 16384 || num_tokens >= (int64_t)1 << 24) return KDACONV_EUNSUPPORTED;
  if (x_stride < 0 || residual_stride < 0) return KDACONV_EUNSUPPORTED;
  // Rows of the residual may not overlap: each is written.
  if (residual != nullptr && num_tokens > 1 && residual_stride < hidden) return KDACONV_EINVAL;
  if (num_tokens == 0) return KDACONV_OK;
  if (!x || !out) return KDACONV_EINVAL;
  if (!element_aligned(x, dtype) || !element_aligned(out, dtype) ||
      !element_aligned(residual, dtype) || !element_aligned(weight, KDACONV_F32))
    return KDACONV_EUNSUPPORTED;
  ResidualNormParams P;
  P.x = static_cast<const char*>(x);
  P.residual = static_cast<char*>(residual);
  P.weight = weight;
  P.out = static_cast<char*>(out);
  P.x_stride = x_stride;
  P.r_stride = residual_stride;
  P.hidden = (int32_t)hidden;
  P.scale = (float)residual_scale;
  P.inv_hidden = (float)(1.0 / (double)hidden);
  P.eps = (float)eps;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == KDACONV_F32)
    launch_residual<kRuleF32>(P, num_tokens, st);
  else if (dtype == KDACONV_F16)
    launch_residual<kRuleF16>(P, num_tokens, st);
  else
    launch_residual<kRuleBF16>(P, num_tokens, st);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}
