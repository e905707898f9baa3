// Expanded attention over packed sequences: the kernel.
//
// For a head of query token i, over the keys t below its reach
//     s_t = scale (q . [k_t, r_t]),  out = sum_t softmax(s)_t v_t
// where r_t, a key's rotated part, is the same for all heads.
//
// A wave holds 32 queries, a workgroup 4 or 8 waves; steps of 64 keys and values go to LDS, one
// ahead of the products. Products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so a lane
// has one query and its softmax needs no other lane but for the largest score; and the scores'
// registers are the second product's right operand as they are: of 16 keys lane half h holds 4 h
// .. 4 h + 3 and 8 + 4 h .., and the left operand takes its keys in that order. That operand is V
// transposed, which LDS delivers (ds_read_b64_tr_b16).
#ifndef KDACONV_EXPANDED_ATTENTION_DEVICE_H_
#define KDACONV_EXPANDED_ATTENTION_DEVICE_H_

#include "attention_device.h"
#include "expanded_attention.h"

namespace kdaconv {

// LDS of a step: 64 keys' own parts, their rotated parts and values, rows of 16-byte chunks.
// Chunk c of row r lies at place c ^ f(r) of its row, with f such that neither 16 rows' chunk
// c (keys) nor chunks 4 i .. 4 i + 3 of 4 rows (values) share a bank.
template <int kDim, int kRope>
struct Step {
  static constexpr int kRow = kDim * 2, kRopeRow = kRope * 2;
  static constexpr int kRopes = kExpandKeys * kRow, kValues = kRopes + kExpandKeys * kRopeRow;
  static constexpr int kBytes = kValues + kExpandKeys * kRow;
  static constexpr int kPer = 64 / (kDim / 8), kRopePer = 64 / (kRope / 8);  // rows per load
  static __device__ __forceinline__ int key_flip(int row) { return kDim == 128 ? row & 15 : (row >> 1) & 7; }
  static __device__ __forceinline__ int rope_flip(int row) { return kRope == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
  static __device__ __forceinline__ int value_flip(int row) { return kDim == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }
};

template <int kF, int kDim, int kRope, int kWaves>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void expanded_kernel(ExpandParams P) {
  using T = Step<kDim, kRope>;
  constexpr int kRows = kWaveRows * kWaves, kThreads = 64 * kWaves;
  constexpr int kOwn = kDim / 16, kAll = kOwn + kRope / 16;  // products per 32 scores
  constexpr int kColumns = kDim / 32;  // blocks of 32 value channels
  __shared__ __attribute__((aligned(16))) char memory[2 * T::kBytes];
  __shared__ int bad[kDim];  // a value channel's first key that is not finite, of those made 0

  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  const int h = lane / 32, n = lane % 32;
  // Long blocks first: they come last in their sequence.
  const int program = P.programs - 1 - (int)(blockIdx.x / (uint32_t)P.heads), head = blockIdx.x % (uint32_t)P.heads;

  // The sequence and block of the program: the largest s with v(s) <= program.
  int s = 0, v = 0;
  for (int stride = P.search_top; stride > 0; stride >>= 6) {
    const int i = s + lane * stride;
    int at = 0;
    bool ok = i < P.seqs;
    if (ok) {
      int a = P.qsl[i];
      a = a < 0 ? 0 : (a > P.tokens ? P.tokens : a);
      at = i + a / kRows;
      ok = at <= program;
    }
    const int found = __builtin_popcountll(__ballot(ok));
    if (found == 0) return;
    s += (found - 1) * stride;
    v = __shfl(at, found - 1);
  }
  s = uniform(s);
  const int block = program - uniform(v);
  const auto bound = [](int x, int low, int high) { return x < low ? low : (x > high ? high : x); };
  const int start = bound(P.qsl[s], 0, P.tokens), rows = bound(P.qsl[s + 1], start, P.tokens) - start;
  const int kstart = bound(P.ksl[s], 0, P.keys), keys = bound(P.ksl[s + 1], kstart, P.keys) - kstart;
  if (block < 0 || block * kRows >= rows) return;

  // What rows see: all keys, or those up to the row's own place, counted from the end.
  const int row = block * kRows + wave * kWaveRows + n;
  const bool live = row < rows;
  const int past = P.causal ? keys - rows + 1 : keys;
  const auto reach_of = [&](int r) { return P.causal ? bound(past + r, 0, keys) : keys; };
  const int reach = reach_of(live ? row : rows - 1);
  const int wave_row = block * kRows + wave * kWaveRows;
  const int least = reach_of(wave_row), most = reach_of(wave_row + kWaveRows < rows ? wave_row + kWaveRows - 1 : rows - 1);
  const int block_least = reach_of(block * kRows);
  const int block_most = reach_of((block + 1) * kRows < rows ? (block + 1) * kRows - 1 : rows - 1);
  const int steps = (block_most + kExpandKeys - 1) / kExpandKeys;

  u32x4 qf[kAll];
  {
    const char* const q = P.q + (int64_t)(start + row) * P.q_ts + (int64_t)head * P.q_hs;
#pragma unroll
    for (int k = 0; k < kAll; ++k) {
      const int c = (k < kOwn ? k : k - kOwn) * 16 + 8 * h;
      const bool there = live && c < (k < kOwn ? P.dim : P.rope);
      qf[k] = *(const u32x4_any*)(there ? q + (k < kOwn ? c : P.dim + c) * 2 : (const char*)kZeros);
    }
#pragma unroll
    for (int k = 0; k < kAll; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[k][i] ^= P.flip;
    // (They arrive here. Else every step would wait for them, and for the step under way.)
#pragma unroll
    for (int k = 0; k < kAll; ++k) asm volatile("" : "+v"(qf[k]));
  }
  for (int i = tid; i < kDim; i += kThreads) bad[i] = INT32_MAX;

  // Where this lane's chunks lie in a load's rows.
  const char* const kb = P.k + (int64_t)kstart * P.k_ts + (int64_t)head * P.k_hs;
  const char* const rb = P.kr + (int64_t)kstart * P.kr_ts;
  const char* const vb = P.v + (int64_t)kstart * P.v_ts + (int64_t)head * P.v_hs;
  constexpr int kChunks = kDim / 8, kRopeChunks = kRope / 8;
  const auto issue = [&](int step) {
    lds_char* const to = (lds_char*)memory + (step & 1) * T::kBytes;
    const int key = step * kExpandKeys;
    constexpr int kLoads = kExpandKeys / T::kPer, kRopeLoads = kExpandKeys / T::kRopePer;
    const bool whole = P.plain && key + kExpandKeys <= keys;
    const int l = (int)fresh(lane);
#pragma unroll
    for (int j = 0; j < (2 * kLoads + kRopeLoads + kWaves - 1) / kWaves; ++j) {
      const int i = wave + j * kWaves;
      if (i < kLoads) {
        const int first = i * T::kPer, r = l / kChunks, c = l % kChunks ^ T::key_flip(first + r);
        const char* const base = kb + (int64_t)(key + first) * P.k_ts;
        const uint32_t offset = r * (uint32_t)P.k_ts + c * 16;
        if (whole)
          to_lds16(base, offset, to + first * T::kRow);
        else
          to_lds16(key + first + r < keys && c * 8 < P.dim ? base + offset : (const char*)kZeros, to + first * T::kRow);
      } else if (i < 2 * kLoads) {
        const int first = (i - kLoads) * T::kPer, r = l / kChunks, c = l % kChunks ^ T::value_flip(first + r);
        const char* const base = vb + (int64_t)(key + first) * P.v_ts;
        const uint32_t offset = r * (uint32_t)P.v_ts + c * 16;
        if (whole)
          to_lds16(base, offset, to + T::kValues + first * T::kRow);
        else
          to_lds16(key + first + r < keys && c * 8 < P.vdim ? base + offset : (const char*)kZeros,
                   to + T::kValues + first * T::kRow);
      } else if (i < 2 * kLoads + kRopeLoads) {
        const int first = (i - 2 * kLoads) * T::kRopePer, r = l / kRopeChunks, c = l % kRopeChunks ^ T::rope_flip(first + r);
        const char* const base = rb + (int64_t)(key + first) * P.kr_ts;
        const uint32_t offset = r * (uint32_t)P.kr_ts + c * 16;
        if (whole)
          to_lds16(base, offset, to + T::kRopes + first * T::kRopeRow);
        else
          to_lds16(key + first + r < keys && c * 8 < P.rope ? base + offset : (const char*)kZeros,
                   to + T::kRopes + first * T::kRopeRow);
      }
    }
  };

  // Operands' places: chunk 2 k + h of key row n (32 more for the second block) ...
  const auto key_operand = [&](const lds_char* step, int b, int k) {
    const int r = (int)n;
    if (k < kOwn) return lds_read16(step + (32 * b + r) * T::kRow + ((2 * k + h) ^ T::key_flip(r)) * 16);
    return lds_read16(step + T::kRopes + (32 * b + r) * T::kRopeRow + ((2 * (k - kOwn) + h) ^ T::rope_flip(r)) * 16);
  };
  // ... and columns 32 c .. of value rows 4 h .. of 16, and of 8 + 4 h .. .
  const int value_row = 4 * h + n % 16 / 4, value_chunk = n / 16 * 2 + n % 4 / 2;
  const auto value_operand = [&](const lds_char* step, int b, int c) {
    const lds_char* const a = step + T::kValues + (16 * b + value_row) * T::kRow +
                              ((4 * c + value_chunk) ^ T::value_flip(value_row)) * 16 + n % 2 * 8;
    const u32x2 x = lds_read_columns(a), y = lds_read_columns(a + 8 * T::kRow);
    return u32x4{x[0], x[1], y[0], y[1]};
  };

  f32x16 O[kColumns];
#pragma unroll
  for (int c = 0; c < kColumns; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[c][i] = 0.0f;
  float top = kLowest, weight = 0.0f;

  if (steps > 0) issue(0);
  for (int step = 0; step < steps; ++step) {
    // This wave's share of the step has arrived; after the barrier everyone's has, and everyone
    // is done with the step before, whose place is free.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (step + 1 < steps) issue(step + 1);
    lds_char* const at = (lds_char*)memory + (step & 1) * T::kBytes;
    const int key = step * kExpandKeys;
    // Rows that do not see a key have weight 0 for it, but 0 times NaN is NaN: where rows differ in
    // what they see, values that are not finite become zeros, and their rows NaN at the end.
    if (block_most != block_least && key + kExpandKeys > block_least) {
      for (int i = tid; i < kExpandKeys * kChunks; i += kThreads) {
        __attribute__((address_space(3))) u32x4* const p = (__attribute__((address_space(3))) u32x4*)(at + T::kValues + i * 16);
        const u32x4 x = *p, y = finite_pairs<kF>(x);
        uint32_t differ = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) differ |= x[j] ^ y[j];
        if (differ != 0) {
          *p = y;
          const int r = i / kChunks, c = (i % kChunks ^ T::value_flip(r)) * 8;
          for (int j = 0; j < 8; ++j)
            if (((x[j / 2] ^ y[j / 2]) >> (j % 2 * 16)) & 0xFFFF) atomicMin(&bad[c + j], key + r);
        }
      }
      lds_barrier();
    }
    if (key >= most) continue;

    f32x16 S[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) S[b][i] = 0.0f;
    // Operands are read a batch ahead of their products.
    constexpr int kBatch = 6, kProducts = 2 * kAll;
    u32x4 a[2][kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) a[0][i] = key_operand(at, i % 2, i / 2);
#pragma unroll
    for (int j = 0; j < kProducts; j += kBatch) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j + kBatch + i < kProducts)
          a[(j / kBatch + 1) % 2][i] = key_operand(at, (j + i) % 2, (j + kBatch + i) / 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j + i < kProducts) S[(j + i) % 2] = mfma_32x32x16<kF>(a[j / kBatch % 2][i], qf[(j + i) / 2], S[(j + i) % 2]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (key + kExpandKeys > least) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[b][i] = key + 32 * b + 8 * (i / 4) + 4 * h + i % 4 < reach ? S[b][i] : -__builtin_huge_valf();
    }
    float high = S[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) high = __builtin_fmaxf(high, S[i / 16][i % 16]);
    high = P.scale * __builtin_fmaxf(high, __shfl_xor(high, 32));
    if (__ballot(high > top + kSlack) != 0) {
      const float next = __builtin_fmaxf(top, high), f = exp2_hw(top - next);
      top = next;
      weight *= f;
#pragma unroll
      for (int c = 0; c < kColumns; ++c) O[c] *= f;
    }
    u32x4 p[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = exp2_hw(__builtin_fmaf(P.scale, S[b / 2][b % 2 * 8 + i], -top));
        weight += x[i];
      }
      p[b] = pack_eight<kF>(x);
    }
    u32x4 y[2][kColumns];
#pragma unroll
    for (int c = 0; c < kColumns; ++c) y[0][c] = value_operand(at, 0, c);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b < 3) {
#pragma unroll
        for (int c = 0; c < kColumns; ++c) y[(b + 1) % 2][c] = value_operand(at, b + 1, c);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < kColumns; ++c) O[c] = mfma_32x32x16<kF>(y[b % 2][c], p[b], O[c]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  weight += __shfl_xor(weight, 32);
  const float f = weight == 0.0f ? 0.0f : 1.0f / weight;
  __syncthreads();  // all values that are not finite are known
  if (!live) return;
  char* const out = P.out + (((int64_t)(start + row) * P.heads + head) * P.vdim) * 2;
#pragma unroll
  for (int c = 0; c < kColumns; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int column = 32 * c + 8 * i + 4 * h;
      if (column >= P.vdim) continue;
      f32x4 x = {f * O[c][4 * i], f * O[c][4 * i + 1], f * O[c][4 * i + 2], f * O[c][4 * i + 3]};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (bad[column + j] < reach) x[j] = __builtin_nanf("");
      Pair<kF>::store(out + column * 2, f32x2{x[0], x[1]});
      Pair<kF>::store(out + column * 2 + 4, f32x2{x[2], x[3]});
    }
}

template <int kF, int kDim, int kRope, int kWaves>
void launch_expanded(const ExpandParams& P, hipStream_t st) {
  hipLaunchKernelGGL((expanded_kernel<kF, kDim, kRope, kWaves>), dim3((unsigned)((int64_t)P.programs * P.heads)),
                     dim3(64 * kWaves), 0, st, P);
}

}  // namespace kdaconv

#endif  // KDACONV_EXPANDED_ATTENTION_DEVICE_H_
