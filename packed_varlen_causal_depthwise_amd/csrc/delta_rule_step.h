// The gated delta rule token by token: the decode step.
//
// One workgroup per (sequence, head), one wave per 32 value columns. A wave holds its
// head_dim x 32 slice of the state in registers for the whole call: lane l owns columns
// 4 (l % 8) .. + 3 of the slice in the head_dim / 8 rows from (head_dim / 8) (l / 8), so
// each load and store instruction moves whole 128-byte pieces of 8 rows. Sums over key
// channels run down the rows in registers and end with three exchanges between lanes.
// The keys, queries and decays of a token do not depend on the state: wave w prepares
// token w of a group of tokens into LDS for all waves, one barrier per group, while the
// state's loads are in flight.
//
// A token costs four FP32 operations per state element against 8 bytes read and written
// for a single-token call, so the state's traffic bounds the decode step. The state passes the
// caches by: between two tokens every other layer's state passes too. 256 sequences of 12
// heads of 128 (403 MB) take 77 us, 5.2 TB/s, after other data went through the caches, and
// 89 with ordinary accesses; only where the state stays in the last-level cache are those
// faster (64 us against 76). A call of 4096 sequences of 1 to 4 tokens, 3 heads of 64: 101 us
// against 115.
#ifndef KDACONV_DELTA_RULE_STEP_H_
#define KDACONV_DELTA_RULE_STEP_H_

#include "delta_rule_device.h"

namespace kdaconv {

template <int kF, int kG, int D>
__global__ __launch_bounds__(2 * D) void delta_rule_step_kernel(const RuleParams P) {
  constexpr int kWaves = D / 32;  // also tokens per group
  constexpr int kRows = D / 8;  // state rows per lane
  constexpr int kEB = elem_bytes<kF>(), kGB = elem_bytes<kG>();
  __shared__ __attribute__((aligned(16))) float sk[2][kWaves][D], sq[2][kWaves][D], sd[2][kWaves][D];
  __shared__ float sb[2][kWaves];

  const int s = blockIdx.x / P.heads, h = blockIdx.x % P.heads;
  const Sequence seq(P, s);
  // (Without tokens a sequence that starts from zeros leaves them.)
  if (seq.len > P.max_len || (seq.len == 0 && (seq.init || seq.line < 0))) return;
  const int wave = uniform(threadIdx.x / kRuleWave), lane = threadIdx.x % kRuleWave;
  const int col = 32 * wave + 4 * (lane % 8), row = kRows * (lane / 8);

  f32x4 S[kRows];
  float* const state = P.states + (seq.line < 0 ? 0 : seq.line) * P.st_line + h * P.st_head +
                       row * D + col;
  if (seq.init) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) S[i] = __builtin_nontemporal_load((const f32x4a4*)(state + i * D));
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) S[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const Gate gate(P, h);
  const int c = 2 * (lane % (D / 2));
  f32x2 bias = {0.0f, 0.0f};
  if (P.dt_bias != nullptr) bias = *(const f32x2a4*)(P.dt_bias + h * D + c);
  const int64_t qk = h / P.share;

  for (int t0 = 0, buf = 0; t0 < seq.len; t0 += kWaves, buf ^= 1) {
    if (t0 + wave < seq.len) {
      const int64_t t = seq.start + t0 + wave;
      const f32x2 kk = Pair<kF>::value(Pair<kF>::load(P.k + (t * P.k_ts + qk * P.k_hs + c) * kEB));
      const f32x2 qq = Pair<kF>::value(Pair<kF>::load(P.q + (t * P.q_ts + qk * P.q_hs + c) * kEB));
      const char* gp = P.g + (t * P.g_ts + h * P.g_hs + c * P.g_cs) * kGB;
      f32x2 gg;
      if (P.g_cs != 0) {
        gg = Pair<kG>::value(Pair<kG>::load(gp));
      } else {
        gg.x = gg.y = load_elem<kG>(gp);
      }
      Factor rk = {1.0f, 0.0f};
      float rq = P.scale;
      if (P.l2_eps >= 0.0f) {
        // (In FP64 the query's square too: in FP32 it would overflow from 2^64 on.)
        const double x = kk.x, y = kk.y, qx = qq.x, qy = qq.y;
        rk = inverse_root(lane_sum<D / 2>(__builtin_fma(x, x, y * y)) + (double)P.l2_eps);
        rq = (float)(P.scale * inverse_root_f64(lane_sum<D / 2>(__builtin_fma(qx, qx, qy * qy)) + (double)P.l2_eps));
      }
      if (lane < D / 2) {
        *(f32x2*)&sk[buf][wave][c] = f32x2{scaled(kk.x, rk), scaled(kk.y, rk)};
        *(f32x2*)&sq[buf][wave][c] = f32x2{qq.x * rq, qq.y * rq};
        f32x2 d[1] = {gg};
        gate.eval(d, bias);
        *(f32x2*)&sd[buf][wave][c] = f32x2{exp2_hw(d[0].x), exp2_hw(d[0].y)};
      }
      if (lane == 0) sb[buf][wave] = beta_value(P, kF, t, h);
    }
    __syncthreads();
    const int n = seq.len - t0 < kWaves ? seq.len - t0 : kWaves;
    for (int w = 0; w < n; ++w) {
      const int64_t t = seq.start + t0 + w;
      const char* vp = P.v + (t * P.v_ts + h * P.v_hs + col) * kEB;
      const f32x2 v0 = Pair<kF>::value(Pair<kF>::load(vp));
      const f32x2 v1 = Pair<kF>::value(Pair<kF>::load(vp + 2 * kEB));
      f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kRows; i += 4) {
        const f32x4 d = *(const f32x4*)&sd[buf][w][row + i];
        const f32x4 k = *(const f32x4*)&sk[buf][w][row + i];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            S[i + e][j] *= d[e];
            y[j] = __builtin_fmaf(S[i + e][j], k[e], y[j]);
          }
      }
      const float b = sb[buf][w];
      f32x4 u, o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = y[j];
        x += __shfl_xor(x, 8);
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
        u[j] = b * ((j < 2 ? v0[j] : v1[j - 2]) - x);
      }
#pragma unroll
      for (int i = 0; i < kRows; i += 4) {
        const f32x4 k = *(const f32x4*)&sk[buf][w][row + i];
        const f32x4 q = *(const f32x4*)&sq[buf][w][row + i];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            S[i + e][j] = __builtin_fmaf(k[e], u[j], S[i + e][j]);
            o[j] = __builtin_fmaf(S[i + e][j], q[e], o[j]);
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] += __shfl_xor(o[j], 8);
        o[j] += __shfl_xor(o[j], 16);
        o[j] += __shfl_xor(o[j], 32);
      }
      if (lane < 8) {
        char* op = P.out + ((t * P.heads + h) * D + col) * kEB;
        Pair<kF>::store(op, f32x2{o[0], o[1]});
        Pair<kF>::store(op + 2 * kEB, f32x2{o[2], o[3]});
      }
    }
  }
  if (seq.line >= 0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) __builtin_nontemporal_store(S[i], (f32x4a4*)(state + i * D));
  }
}

template <int kF, int kG>
void launch_rule_step(const RuleParams& P, int head_dim, hipStream_t st) {
  const dim3 grid((unsigned)(P.num_seqs * (int64_t)P.heads));
  if (head_dim == 128)
    hipLaunchKernelGGL((delta_rule_step_kernel<kF, kG, 128>), grid, dim3(256), 0, st, P);
  else
    hipLaunchKernelGGL((delta_rule_step_kernel<kF, kG, 64>), grid, dim3(128), 0, st, P);
}

}  // namespace kdaconv

#endif  // KDACONV_DELTA_RULE_STEP_H_
