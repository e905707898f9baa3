// Expanded attention over packed sequences: the kernel.
//
// For a head of query token i, over the keys t below its reach
//     s_t = scale (q . [k_t, r_t]),  out = sum_t softmax(s)_t v_t
// where r_t, a key's rotated part, is the same for all heads.
//
// A wave holds 32 queries, a workgroup 4 or 8 waves; steps of 64 keys and values go to LDS ahead of
// the products. Of 8 waves two share each SIMD, and the matrix unit and the vector unit would
// take turns if they kept step: both products, then both softmaxes. So waves 4 to 7 run half a
// step behind: while one wave of a SIMD multiplies (values of the last step, keys of the next),
// the other one weighs its scores. Barriers keep them so. One prompt of 16384 tokens, 12 heads of
// 128 + 64 channels, takes 925 to 970 us so from card to card (1115 to 1065 TFLOP/s, where a library
// product of 8192^3 reaches 1242), and 1067 in step where it took 925. The matrix unit is busy 62% of
// the time, at the clock that its power leaves. Products are taken transposed, S^T = K Q^T and O^T =
// V^T P^T, so a lane
// has one query and its softmax needs no other lane but for the largest score; and the scores'
// registers are the second product's right operand as they are: of 16 keys lane half h holds 4 h
// .. 4 h + 3 and 8 + 4 h .., and the left operand takes its keys in that order. That operand is V
// transposed, which LDS delivers (ds_read_b64_tr_b16).
#ifndef KDACONV_EXPANDED_ATTENTION_DEVICE_H_
#define KDACONV_EXPANDED_ATTENTION_DEVICE_H_

#include "attention_device.h"
#include "expanded_attention.h"

namespace kdaconv {

// LDS of a step: 64 keys' own parts, their rotated parts and values, rows of 16-byte chunks. A load
// fills 1 KB, rows in a row; chunk c of row r lies at place c ^ f(r) of its row, and between loads'
// pieces of keys lie a chunk or two. f and the gaps are such that neither 16 rows' chunk c (keys)
// nor chunks 4 i .. 4 i + 3 of 4 rows (values) share a bank, and f changes few bits of c: what it
// leaves alone is a constant in an address.
// Pieces of 4 rows (128 channels) lie a chunk further apart each; of 8 rows (64 channels, two rows
// to a period of the banks) two chunks in every pair, and pairs at that period; of 16 as they are.
__host__ __device__ constexpr int piece(int channels, int i) {
  return channels == 128 ? i * 1040 : channels == 64 ? i / 2 * 2304 + i % 2 * 1056 : i * 1024;
}

template <int kDim, int kRope>
struct Step {
  static constexpr int kRow = kDim * 2, kRopeRow = kRope * 2;
  static constexpr int kPer = 64 / (kDim / 8), kRopePer = 64 / (kRope / 8);  // rows per load
  static constexpr int kRopes = piece(kDim, kExpandKeys / kPer), kKeyBytes = kRopes + piece(kRope, kExpandKeys / kRopePer);
  static constexpr int kValueBytes = kExpandKeys * kRow;
  static __device__ __forceinline__ int eight_flip(int row) { return ((row >> 1) & 1) | ((row >> 2) & 1) << 2; }
  static __device__ __forceinline__ int key_flip(int row) { return kDim == 128 ? (row & 3) << 2 : eight_flip(row); }
  static __device__ __forceinline__ int rope_flip(int row) { return kRope == 64 ? eight_flip(row) : (row >> 2) & 3; }
  static __device__ __forceinline__ int value_flip(int row) { return kDim == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }
  // Where a row begins.
  static __device__ __forceinline__ constexpr int key_row(int row) { return piece(kDim, row / kPer) + row % kPer * kRow; }
  static __device__ __forceinline__ constexpr int rope_row(int row) {
    return kRopes + piece(kRope, row / kRopePer) + row % kRopePer * kRopeRow;
  }
  // Products that share an address register: chunks 2 k and 2 (k + 1), k even, but for 32 channels.
  static constexpr int kShare = 2, kRopeShare = kRope == 64 ? 2 : 1;
};

// In the place of a row's weight in a part of the keys of which it sees none. (Where it sees one of
// score -inf the weight is 0, but 0 times its value may be NaN.)
constexpr float kUnseen = -1.0f;

// The sequence and block of a program: the largest s with v(s) <= program.
template <int kRows>
__device__ __forceinline__ bool find_program(const ExpandParams& P, int program, int lane, int& sequence, int& block) {
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
    if (found == 0) return false;
    s += (found - 1) * stride;
    v = __shfl(at, found - 1);
  }
  sequence = uniform(s);
  block = program - uniform(v);
  return block >= 0;
}

template <int kF, int kDim, int kRope, int kWaves>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(kWaves / 4, kWaves / 4))) void expanded_kernel(ExpandParams P) {
  using T = Step<kDim, kRope>;
  constexpr int kRows = kWaveRows * kWaves, kThreads = 64 * kWaves;
  constexpr int kOwn = kDim / 16, kAll = kOwn + kRope / 16;  // products per 32 scores
  constexpr int kColumns = kDim / 32;  // blocks of 32 value channels
  constexpr int kPlaces = 3;  // of steps' keys, and of their values
  __shared__ __attribute__((aligned(16))) char memory[kPlaces * (T::kKeyBytes + T::kValueBytes)];
  __shared__ int bad[kDim];  // a value channel's first key that is not finite, of those made 0

  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  const int h = lane / 32, n = lane % 32;
  // Long blocks first: they come last in their sequence.
  const int program = P.programs - 1 - (int)(blockIdx.x / (uint32_t)P.heads), head = blockIdx.x % (uint32_t)P.heads;

  int s, block;
  if (!find_program<kRows>(P, program, lane, s, block)) return;
  const auto bound = [](int x, int low, int high) { return x < low ? low : (x > high ? high : x); };
  const int start = bound(P.qsl[s], 0, P.tokens), rows = bound(P.qsl[s + 1], start, P.tokens) - start;
  int kstart = bound(P.ksl[s], 0, P.keys), keys = bound(P.ksl[s + 1], kstart, P.keys) - kstart;
  if (block * kRows >= rows) return;

  // What rows see: all keys, or those up to the row's own place, counted from the end.
  const int row = block * kRows + wave * kWaveRows + n;
  const bool live = row < rows;
  int past = P.causal ? keys - rows + 1 : keys;
  const auto reach_of = [&](int r) { return P.causal ? bound(past + r, 0, keys) : keys; };
  if (P.splits > 1) {
    // This workgroup's part of the block's keys, as though they were all.
    const int end = reach_of((block + 1) * kRows < rows ? (block + 1) * kRows - 1 : rows - 1);
    const int64_t all = (end + kExpandKeys - 1) / kExpandKeys;
    const int from = (int)(all * blockIdx.y / P.splits) * kExpandKeys, to = (int)(all * (blockIdx.y + 1) / P.splits) * kExpandKeys;
    kstart += from;
    past -= from;
    keys = (to < keys ? to : keys) - from;
  }
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
      qf[k] = *(Global<u32x4_any>)(there ? q + (k < kOwn ? c : P.dim + c) * 2 : (const char*)kZeros);
    }
#pragma unroll
    for (int k = 0; k < kAll; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[k][i] ^= P.flip;
    // A scale of 0 is taken by the queries: the scores of keys that are not seen are -inf, and that
    // times 0 would be NaN. (Elements that are not finite become NaN: their exponent's last bit
    // moves to the mantissa's first.)
    if (P.vanish) {
      constexpr uint32_t kLast = kF == kRuleBF16 ? 0x00800080u : 0x04000400u;
#pragma unroll
      for (int k = 0; k < kAll; ++k) {
        qf[k] ^= finite_pairs<kF>(qf[k]);
        qf[k] |= (qf[k] & kLast) >> 1;
      }
    }
    // (They arrive here. Else every step would wait for them, and for the step under way.)
#pragma unroll
    for (int k = 0; k < kAll; ++k) asm volatile("" : "+v"(qf[k]));
  }
  for (int i = tid; i < kDim; i += kThreads) bad[i] = INT32_MAX;
  // The values before the first.
  for (int i = tid; i < T::kValueBytes / 16; i += kThreads)
    *(u32x4*)(memory + sizeof memory - T::kValueBytes + i * 16) = u32x4{0, 0, 0, 0};

  // Where this lane's chunks lie in a load's rows.
  const char* const kb = P.k + (int64_t)kstart * P.k_ts + (int64_t)head * P.k_hs;
  const char* const rb = P.rope > 0 ? P.kr + (int64_t)kstart * P.kr_ts : kb;
  const char* const vb = P.v + (int64_t)kstart * P.v_ts + (int64_t)head * P.v_hs;
  constexpr int kChunks = kDim / 8, kRopeChunks = kRope / 8;
  lds_char* const key_ring = (lds_char*)memory;
  lds_char* const value_ring = key_ring + kPlaces * T::kKeyBytes;
  // This wave's loads of a step: first of values, then of keys, then of rotated parts. A lane's
  // place in each kind's rows and channels; a channel that is missing reads the first ones (queries
  // are zero there, and no sum is taken), and so does a rotated part.
  constexpr int kLoads = kExpandKeys / T::kPer / kWaves, kRopeLoads = kExpandKeys / T::kRopePer;
  constexpr int kTurns = 2 * kLoads + (kRopeLoads + kWaves - 1) / kWaves, kSure = 2 * kLoads + kRopeLoads / kWaves;
  const int load_row = wave * T::kPer + lane / kChunks, rope_row = wave * T::kRopePer + lane / kRopeChunks;
  const auto channel = [](int c, int channels) { return c * 8 < channels ? c * 16u : 0u; };
  const uint32_t value_channel = channel(lane % kChunks ^ T::value_flip(load_row), P.vdim);
  const uint32_t key_channel = channel(lane % kChunks ^ T::key_flip(load_row), P.dim);
  const uint32_t rope_channel = channel(lane % kRopeChunks ^ T::rope_flip(rope_row), P.rope);
  static_assert(T::kPer * kWaves % 16 == 0 && T::kRopePer * kWaves % 16 == 0, "a wave's rows flip alike");
  // Load j of step `step`'s values, to place `place`, or of the next step's keys, to the next place.
  // Past the last key that key comes again: its scores are masked, and clean() sees to its values.
  const auto issue = [&](int step, int place, int j) {
    const bool value = j < kLoads, rope = j >= 2 * kLoads;
    const int turn = (value ? j : rope ? j - 2 * kLoads : j - kLoads) * kWaves;  // loads before, of all waves
    if (rope && wave + turn >= kRopeLoads) return;
    int key = (value ? step : step + 1) * kExpandKeys;
    key = key < keys ? key : keys - 1;
    const int next = place + 1 == kPlaces ? 0 : place + 1;
    const int64_t stride = value ? P.v_ts : rope ? P.kr_ts : P.k_ts;
    const int first = turn * (rope ? T::kRopePer : T::kPer);
    int row = first + (int)fresh(rope ? rope_row : load_row);
    row = row < keys - key ? row : keys - 1 - key;
    lds_char* const to = value ? value_ring + place * T::kValueBytes + (first + wave * T::kPer) * T::kRow
                         : rope ? key_ring + next * T::kKeyBytes + T::kRopes + piece(kRope, turn + wave)
                                : key_ring + next * T::kKeyBytes + piece(kDim, turn + wave);
    to_lds16((value ? vb : rope ? rb : kb) + key * stride,
             __umul24(row, (uint32_t)stride) + (value ? value_channel : rope ? rope_channel : key_channel), to);
  };

  // Operands' places in LDS, of the step that is next: chunk 2 k + h of key row n, for channels of
  // its own and rotated ones (32 rows on for the second block) ...
  constexpr int kOwnBases = kOwn / T::kShare, kRopeBases = kRope / 16 / T::kRopeShare;
  const lds_char* key_at[kOwnBases];
  const lds_char* rope_at[kRopeBases];
#pragma unroll
  for (int k = 0; k < kOwnBases; ++k)
    key_at[k] = key_ring + T::key_row(n) + ((2 * T::kShare * k + h) ^ T::key_flip(n)) * 16;
#pragma unroll
  for (int k = 0; k < kRopeBases; ++k)
    rope_at[k] = key_ring + T::rope_row(n) + ((2 * T::kRopeShare * k + h) ^ T::rope_flip(n)) * 16;
  // ... and columns 32 c .. of value rows 4 h .. of 16, and of 8 + 4 h .., of the step before.
  const lds_char* value_at[kColumns];
  {
    const int row = 4 * h + n % 16 / 4, chunk = n / 16 * 2 + n % 4 / 2;
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
      value_at[c] = value_ring + (kPlaces - 1) * T::kValueBytes + row * T::kRow +
                    ((4 * c + chunk) ^ T::value_flip(row)) * 16 + n % 2 * 8;
  }
  const auto move_on = [&](int place) {  // from `place` of the keys to the next
    const int keys_by = (place + 1 == kPlaces ? 1 - kPlaces : 1) * T::kKeyBytes;
    const int values_by = (place == 0 ? 1 - kPlaces : 1) * T::kValueBytes;
#pragma unroll
    for (int k = 0; k < kOwnBases; ++k) key_at[k] += keys_by;
#pragma unroll
    for (int k = 0; k < kRopeBases; ++k) rope_at[k] += keys_by;
#pragma unroll
    for (int c = 0; c < kColumns; ++c) value_at[c] += values_by;
  };
  const auto key_operand = [&](int b, int k) {
    const int r = k - kOwn;  // (32 rows are whole pieces)
    return k < kOwn ? lds_read16(key_at[k / T::kShare] + k % T::kShare * 32 + T::key_row(32) * b)
                    : lds_read16(rope_at[r / T::kRopeShare] + r % T::kRopeShare * 32 + (T::rope_row(32) - T::kRopes) * b);
  };
  const auto value_operand = [&](int b, int c) {
    const u32x2 x = lds_read_columns(value_at[c] + 16 * b * T::kRow);
    const u32x2 y = lds_read_columns(value_at[c] + (16 * b + 8) * T::kRow);
    return u32x4{x[0], x[1], y[0], y[1]};
  };

  f32x16 O[kColumns];
#pragma unroll
  for (int c = 0; c < kColumns; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[c][i] = 0.0f;
  float top = kLowest, weight = 0.0f;

  f32x16 S[2];
  u32x4 p[4] = {};

  // Values of step `step - 1`, then keys of step `step`. The products' left operands are one stream,
  // read kAhead batches ahead: four waves at once take from LDS all that it gives.
  const auto multiply = [&](int step) {
    __builtin_amdgcn_s_setprio(1);  // the products wait for nothing that the other wave does
    constexpr int kValueProducts = 4 * kColumns, kProducts = kValueProducts + 2 * kAll, kBatch = 2, kAhead = 3;
    // Operand i: values' block and columns, or block and channels of keys.
    const auto operand = [&](int i) {
      return i < kValueProducts ? value_operand(i / kColumns, i % kColumns)
                                : key_operand((i - kValueProducts) % 2, (i - kValueProducts) / 2);
    };
    constexpr int kBatches = kProducts / kBatch;
    // Once more after a wave's last step, for its values: a second loop without keys would cost
    // more registers than there are, and the scores are not looked at. Of step 0's values, those
    // before the first, weights are 0.
    if ((step - 1) * kExpandKeys < most) {
      u32x4 a[kAhead + 1][kBatch];
#pragma unroll
      for (int g = 0; g < kAhead; ++g)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) a[g][i] = operand(g * kBatch + i);
#pragma unroll
      for (int g = 0; g < kBatches; ++g) {
        if (g + kAhead < kBatches) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) a[(g + kAhead) % (kAhead + 1)][i] = operand((g + kAhead) * kBatch + i);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int k = g * kBatch + i, j = k - kValueProducts;
          if (k < kValueProducts)
            O[k % kColumns] = mfma_32x32x16<kF>(a[g % (kAhead + 1)][i], p[k / kColumns], O[k % kColumns]);
          else
            S[j % 2] = mfma_32x32x16<kF>(a[g % (kAhead + 1)][i], qf[j / 2], j < 2 ? f32x16{} : S[j % 2]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
  };

  // The scores of step `step`, whose keys lie in place `place`, become weights. And the loads for
  // the steps to come go out, which between products would hold those up (LDS takes 1 KB in some
  // 45 cycles at best).
  const auto weigh = [&](int step, int place) {
#pragma unroll
    for (int j = 0; j < kTurns; ++j) issue(step + 1, place + 1 == kPlaces ? 0 : place + 1, j);
    const int key = step * kExpandKeys;
    if (key >= most) return;
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
  };

  // Rows that do not see a key have weight 0 for it, but 0 times NaN is NaN: where rows differ in
  // what they see, values that are not finite become zeros, and rows that see one get NaN in that
  // channel at the end. And where keys end the last one's values stand for missing ones.
  const auto clean = [&](int step, int place) {
    const int key = step * kExpandKeys;
    if (key + kExpandKeys <= (block_most == block_least ? keys : block_least)) return;
    for (int i = tid; i < kExpandKeys * kChunks; i += kThreads) {
      __attribute__((address_space(3))) u32x4* const at =
          (__attribute__((address_space(3))) u32x4*)(value_ring + place * T::kValueBytes + i * 16);
      const u32x4 x = *at, y = finite_pairs<kF>(x);
      uint32_t differ = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) differ |= x[j] ^ y[j];
      if (differ != 0) {
        *at = y;
        const int r = i / kChunks, c = (i % kChunks ^ T::value_flip(r)) * 8;
        for (int j = 0; j < 8; ++j)
          if (((x[j / 2] ^ y[j / 2]) >> (j % 2 * 16)) & 0xFFFF) atomicMin(&bad[c + j], key + r);
      }
    }
    lds_barrier();
  };

  // Times are counted in phases, with a barrier between any two. Waves ahead multiply for step t
  // in phase 2 t and weigh in 2 t + 1, those behind a phase later. Step t's keys are read in
  // phases 2 t and 2 t + 1, its values in 2 t + 2 and 2 t + 3. A wave that weighs step t sends for
  // step t + 2's keys and step t + 1's values, to places last read in phase 2 t - 1, and all wait
  // for them at the end of phase 2 t + 3: waves ahead when they have sent for more, those behind
  // before.
  const bool behind = kWaves == 8 && wave >= 4;
  if (steps > 0) {
#pragma unroll
    for (int j = kLoads; j < kTurns; ++j) issue(-1, kPlaces - 1, j);
#pragma unroll
    for (int j = 0; j < kTurns; ++j) issue(0, 0, j);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (behind) lds_barrier();
    int place = 0;
    for (int step = 0; step < steps; ++step) {
      if (!behind && step > 0) clean(step - 1, place == 0 ? kPlaces - 1 : place - 1);
      multiply(step);
      if (behind) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
      if (behind) clean(step, place);
      weigh(step, place);
      if (!behind) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kSure) : "memory");
      lds_barrier();
      move_on(place);
      place = place + 1 == kPlaces ? 0 : place + 1;
    }
    if (!behind && steps > 0) clean(steps - 1, place == 0 ? kPlaces - 1 : place - 1);
    multiply(steps);
    if (kWaves == 8 && !behind) lds_barrier();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads of steps past the end
  }

  weight += __shfl_xor(weight, 32);
  const float f = weight == 0.0f ? 0.0f : 1.0f / weight;
  __syncthreads();  // all values that are not finite are known
  if (!live) return;
  if (P.splits > 1) {
    const ExpandPartial part{kRows, P.vdim};
    float* const mine = P.partial + part.floats() * (((int64_t)program * P.heads + head) * P.splits + blockIdx.y);
    const int r = wave * kWaveRows + n;
    if (h == 0) {
      mine[part.exponent() + r] = top;
      mine[part.weight() + r] = reach > 0 ? weight : kUnseen;
    }
    if (reach <= 0) return;  // (its sums are not looked at)
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int column = 32 * c + 8 * i + 4 * h;
        if (column >= P.vdim) continue;
        f32x4 x = {O[c][4 * i], O[c][4 * i + 1], O[c][4 * i + 2], O[c][4 * i + 3]};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (bad[column + j] < reach) x[j] = __builtin_nanf("");
        *(f32x4*)(mine + (int64_t)r * P.vdim + column) = x;
      }
    return;
  }
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

// Joins the parts of a block's keys: a workgroup per block and head, 8 channels of a row at a time.
constexpr int kExpandJoinThreads = 256;

template <int kF, int kRows>
__global__ __launch_bounds__(kExpandJoinThreads) void expanded_join_kernel(ExpandParams P) {
  const int tid = threadIdx.x, head = blockIdx.x % (uint32_t)P.heads, program = blockIdx.x / (uint32_t)P.heads;
  int s, block;
  if (!find_program<kRows>(P, program, tid % 64, s, block)) return;
  const auto bound = [](int x, int low, int high) { return x < low ? low : (x > high ? high : x); };
  const int start = bound(P.qsl[s], 0, P.tokens), all = bound(P.qsl[s + 1], start, P.tokens) - start;
  const int rows = all - block * kRows < kRows ? all - block * kRows : kRows, chunks = P.vdim / 8;
  const ExpandPartial part{kRows, P.vdim};
  const float* const parts = P.partial + part.floats() * ((int64_t)blockIdx.x * P.splits);
  for (int i = blockIdx.y * kExpandJoinThreads + tid; i < rows * chunks; i += kExpandJoinThreads * gridDim.y) {
    const int r = (int)((uint32_t)i / (uint32_t)chunks), c = i - r * chunks;
    float high = kLowest, total = 0.0f;
    for (int k = 0; k < P.splits; ++k) {
      const float* const p = parts + part.floats() * k;
      high = __builtin_fmaxf(high, p[part.exponent() + r]);  // (the lowest, of a part without weight)
    }
    f32x4 v[2] = {};
    for (int k = 0; k < P.splits; ++k) {
      const float* const p = parts + part.floats() * k;
      const float l = p[part.weight() + r];
      if (l == kUnseen) continue;
      const float f = exp2_hw(p[part.exponent() + r] - high);
      const f32x4* const q = (const f32x4*)(p + (int64_t)r * P.vdim + c * 8);
      total = __builtin_fmaf(f, l, total);
      v[0] += f * q[0];
      v[1] += f * q[1];
    }
    const float f = total == 0.0f ? 0.0f : 1.0f / total;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = f * v[j / 4][j % 4];
    store_eight<kF>(P.out + ((((int64_t)start + block * kRows + r) * P.heads + head) * P.vdim + c * 8) * 2, o);
  }
}

template <int kF, int kDim, int kRope, int kWaves>
void launch_expanded(const ExpandParams& P, hipStream_t st) {
  const unsigned blocks = (unsigned)((int64_t)P.programs * P.heads);
  hipLaunchKernelGGL((expanded_kernel<kF, kDim, kRope, kWaves>), dim3(blocks, P.splits), dim3(64 * kWaves), 0, st, P);
  if (P.splits > 1)
    hipLaunchKernelGGL((expanded_join_kernel<kF, kWaveRows * kWaves>), dim3(blocks, kWaves), dim3(kExpandJoinThreads), 0, st, P);
}

}  // namespace kdaconv

#endif  // KDACONV_EXPANDED_ATTENTION_DEVICE_H_
