// Absorbed latent attention over the paged cache: the kernels.
//
// For a row (a head of a new token) with query (ql, qr) and the cached tokens t below its reach
//     s_t = scale (ql . c_t + qr . r_t),  out = sum_t softmax(s)_t c_t
// so a token's latent is key and value at once: it goes to LDS once and is read there twice.
//
// Products are taken transposed, S^T = K Q^T and O^T = C^T P^T. A matrix product leaves a lane
// with one column, here one query: its softmax needs no other lane but for the largest score,
// and the scores are in place as the second product's right operand. (Of 32 keys lane group g
// holds 4 g .. 4 g + 3 and 16 + 4 g .. ; the left operand takes its keys in that order.) That
// operand is C transposed, which LDS delivers: ds_read_b64_tr_b16 hands 16 lanes the columns of
// 4 rows of 16.
#ifndef KDACONV_LATENT_ATTENTION_DEVICE_H_
#define KDACONV_LATENT_ATTENTION_DEVICE_H_

#include "latent_attention.h"
#include "latent_device.h"

namespace kdaconv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int kF>
__device__ __forceinline__ f32x4 mfma_16x16x32(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kF == kRuleBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0, 0, 0);
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

// 16 bytes per lane from memory to LDS, at the wave's place + 16 times the lane's number.
__device__ __forceinline__ void to_lds16(const char* from, lds_char* wave_to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)wave_to, 16, 0, 0);
}

// Hides that x is the same in every iteration of a loop. Without it the compiler works out
// all rows' offsets before the loop, and spills them.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Scheduling of n products and the LDS reads of one operand each (of two halves each): some
// reads ahead, then one for each product. Left alone the compiler waits for every read.
template <int kN, int kAhead = 8>
__device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int i = 0; i < kN - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
}

template <int kN, int kAhead = 6>
__device__ __forceinline__ void interleave_pairs() {
  __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAhead, 0);
#pragma unroll
  for (int i = 0; i < kN - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
}

// Pairs of elements with 0 in the place of infinities and NaN.
template <int kF>
__device__ __forceinline__ u32x2 finite_pairs(u32x2 x) {
  constexpr uint32_t kHigh = kF == kRuleBF16 ? 0x7F800000u : 0x7C000000u, kLow = kHigh >> 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if ((x[i] & kHigh) == kHigh) x[i] &= 0xFFFFu;
    if ((x[i] & kLow) == kLow) x[i] &= 0xFFFF0000u;
  }
  return x;
}

// What a key outside the sequence, and channels past a latent's, read.
static __device__ const uint32_t kZeros[kLatentMax / 2] = {};

// A place on the line of work: sequence, block of rows, tile of keys.
struct Place {
  int s, b, t;
  __device__ bool before(const Place& o) const { return s < o.s || (s == o.s && (b < o.b || (b == o.b && t < o.t))); }
};

template <int kRows, int kIter>
struct Line {
  // The rows, keys and units of a sequence. Offsets out of order or out of range give a
  // sequence without rows.
  static __device__ __forceinline__ int tokens(const AttendParams& P, int s, int& start) {
    if (P.qsl == nullptr) {
      start = s;
      return 1;
    }
    int a = P.qsl[s], b = P.qsl[s + 1];
    a = a < 0 ? 0 : (a > P.tokens ? P.tokens : a);
    b = b < a ? a : (b > P.tokens ? P.tokens : b);
    start = a;
    return b - a;
  }
  static __device__ __forceinline__ int keys(const AttendParams& P, int s) {
    int64_t most = (int64_t)P.T.width * P.C.page_size.d;
    most = most < kMostKeys ? most : kMostKeys;
    const int n = P.seq_lens[s];
    return n < 0 ? 0 : (n > most ? (int)most : n);
  }
  static __device__ __forceinline__ int blocks(const AttendParams& P, int tokens) {
    return (int)(((int64_t)tokens * P.heads.d + kRows - 1) / kRows);
  }
  static __device__ __forceinline__ int tiles(int keys) { return (int)(((int64_t)keys + kIter - 1) / kIter); }
  static __device__ __forceinline__ int64_t units(const AttendParams& P, int s) {
    int start;
    const int n = tokens(P, s, start);
    return n > 0 ? (int64_t)blocks(P, n) * (tiles(keys(P, s)) + kBlockUnits) : 0;
  }
};

// Finds this worker's part of the line. All threads of the workgroup call it; `room` is LDS of
// 128 bytes. Returns the number of workers that have a part.
template <int kRows, int kIter>
__device__ __forceinline__ int find_part(const AttendParams& P, char* room, Place& from, Place& to, int64_t& all) {
  using L = Line<kRows, kIter>;
  int64_t* const sums = (int64_t*)room;  // per wave
  int* const found = (int*)(room + 64);  // from, to
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  constexpr int kThreads = 64 * kAttendWaves;
  int64_t mine = 0;
  for (int s = tid; s < P.seqs; s += kThreads) mine += L::units(P, s);
  mine = lane_sum<64>(mine);
  if (lane == 0) sums[wave] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kAttendWaves; ++i) total += sums[i];
  all = total;
  int64_t workers = total / kLeastUnits;
  workers = workers < 1 ? 1 : (workers > P.workers ? P.workers : workers);
  const int w = blockIdx.x;
  if (w >= workers || total == 0) return (int)workers;
  const int64_t lo = total * w / workers, hi = total * (w + 1) / workers;
  if (tid < 6) found[tid] = tid % 3 == 0 ? P.seqs : 0;
  int64_t before = 0;
  for (int base = 0; base < P.seqs && before <= hi; base += kThreads) {
    const int s = base + tid;
    const int64_t u = s < P.seqs ? L::units(P, s) : 0;
    int64_t run = u;  // inclusive running sum
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t other = __shfl_up(run, d);
      run += lane >= d ? other : 0;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    int64_t first = before, chunk = 0;
#pragma unroll
    for (int i = 0; i < kAttendWaves; ++i) {
      if (i < wave) first += sums[i];
      chunk += sums[i];
    }
    first += run - u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t at = e == 0 ? lo : hi;
      if (at >= first && at < first + u) {
        const int tiles = L::tiles(L::keys(P, s)), per = tiles + kBlockUnits;
        const int64_t off = at - first;
        const int b = (int)(off / per), r = (int)(off - (int64_t)b * per);
        found[3 * e] = s;
        found[3 * e + 1] = b;
        found[3 * e + 2] = r > kBlockUnits ? r - kBlockUnits : 0;
      }
    }
    before += chunk;
  }
  __syncthreads();
  from = Place{uniform(found[0]), uniform(found[1]), uniform(found[2])};
  to = Place{uniform(found[3]), uniform(found[4]), uniform(found[5])};
  __syncthreads();
  return (int)workers;
}

// LDS of one tile: 32 latents, then 32 rotated parts, rows of 16-byte chunks. Chunk c of row r
// lies at place c ^ f(r) of its row, with f such that neither 16 rows' chunk c (the products'
// left operand) nor chunks 2 i, 2 i + 1 of 8 rows (columns) share a bank.
template <int kLatent>
struct Tile {
  static constexpr int kRow = kLatent * 2, kRope = kRopeMax * 2;
  static constexpr int kRopes = kTileKeys * kRow;
  static constexpr int kBytes = kRopes + kTileKeys * kRope;
  static __device__ __forceinline__ int latent_flip(int row) { return ((row & 7) << 1) | ((row >> 3) & 1); }
  static __device__ __forceinline__ int rope_flip(int row) { return (row >> 1) & 7; }
};

// One tile on its way: keys' addresses, and for 8 bits the codes in registers.
template <int kF, int kLatent, int kQ, bool kE4m3>
struct Loader {
  using T = Tile<kLatent>;
  static constexpr int kChunks = kLatent / 8;  // 16-byte chunks of 16-bit elements per row
  static constexpr int kLatentLoads = kE4m3 ? kTileKeys * (kLatent / 16) / 64 / kQ : kTileKeys * kChunks / 64 / kQ;
  static constexpr int kRopeLoads = kTileKeys / 8 / kQ;  // 8 rows each
  static constexpr int kScaleLoads = kE4m3 ? kLatentLoads : 1;

  int window = -1;  // page of number window_at + lane of the sequence
  int window_at = 0, window_of = -1;  // the sequence
  const char* lat;  // of key `lane % 32`; zeros where there is none
  const char* rop;
  const uint8_t* sc;
  uint32_t mask;  // keys that are there

  u32x4 codes[kE4m3 ? kLatentLoads : 1];
  uint32_t scales[kScaleLoads];
  u32x4 ropes[kE4m3 ? kRopeLoads : 1];

  // Finds the keys from `first` on. The lanes hold a window of the page table: loads return in
  // order, so an entry loaded for each tile would wait for all tiles under way.
  __device__ __forceinline__ void find(const AttendParams& P, int s, int first, int keys, int lane) {
    lane = (int)fresh(lane);
    const int end = first + kTileKeys < keys ? first + kTileKeys : keys;
    const int low = (int)P.C.page_size((uint32_t)first);
    if (window_of != s || (end > first && (int)P.C.page_size((uint32_t)(end - 1)) >= window_at + 64)) {
      window_of = s;
      window_at = low;
      window = low + lane < P.T.width ? P.T.table[s * P.T.stride + low + lane] : -1;
    }
    const int key = first + lane % kTileKeys;
    const uint32_t p = P.C.page_size((uint32_t)key);
    const int at = key - (int)(p * P.C.page_size.d);
    const int page = __shfl(window, (int)p - window_at);
    const bool ok = key < keys && page >= 0 && page < P.C.num_pages;
    mask = (uint32_t)__ballot(ok);
    lat = ok ? P.C.latents + page * P.C.lat_page + at * P.C.lat_slot : (const char*)kZeros;
    rop = ok ? P.C.ropes + page * P.C.rope_page + at * P.C.rope_slot : (const char*)kZeros;
    if constexpr (kE4m3) sc = ok ? P.C.scales + page * P.C.scale_page + at * P.C.scale_slot : (const uint8_t*)kZeros;
  }

  template <class X>
  static __device__ __forceinline__ X* row_of(X* p, int row) {
    const uint64_t a = (uint64_t)p;
    const uint32_t lo = __shfl((uint32_t)a, row), hi = __shfl((uint32_t)(a >> 32), row);
    return (X*)(((uint64_t)hi << 32) | lo);
  }
  // The same for a row that all lanes want.
  static __device__ __forceinline__ const char* row_uniform(const char* p, int row) {
    const uint64_t a = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)a, row), hi = __builtin_amdgcn_readlane((uint32_t)(a >> 32), row);
    return (const char*)(((uint64_t)hi << 32) | lo);
  }

  // Sends the tile on its way: 16 bits straight to LDS, 8 bits to registers. `part` of the
  // kQ waves that share it takes its rows.
  __device__ __forceinline__ void issue(const AttendParams& P, lds_char* to, int part, int lane) {
    lane = (int)fresh(lane);
    if constexpr (!kE4m3) {
      constexpr int kPer = 64 / kChunks;  // rows per load
      // Flips reach 16 chunks. Where a latent's end is at a multiple of them its lanes are told
      // by their number alone: those past it read its first chunks (queries are zero there, and
      // no output is taken).
      if (P.C.latent % 128 == 0) {
        const int c = lane % kChunks;
        const uint32_t at = (c * 8 < P.C.latent ? c : c % 16) * 16;
#pragma unroll
        for (int i = 0; i < kLatentLoads; ++i) {
          const int first = (part * kLatentLoads + i) * kPer;
          if constexpr (kPer == 1) {
            to_lds16(row_uniform(lat, first) + (at ^ (T::latent_flip(first) * 16)), to + first * T::kRow);
          } else {
            const int row = first + lane / kChunks;
            to_lds16(row_of(lat, row) + (at ^ (T::latent_flip(row) * 16)), to + first * T::kRow);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLatentLoads; ++i) {
          const int first = (part * kLatentLoads + i) * kPer, row = first + lane / kChunks;
          const char* const base = row_of(lat, row);
          const int c = (lane % kChunks) ^ T::latent_flip(row);
          to_lds16(c * 8 < P.C.latent ? base + c * 16 : (const char*)kZeros, to + first * T::kRow);
        }
      }
      if (P.C.rope > 0) {
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
          const int first = (part * kRopeLoads + i) * 8, row = first + lane / 8;
          const char* const base = row_of(rop, row);
          const int c = (lane % 8) ^ T::rope_flip(row);
          to_lds16(c * 8 < P.C.rope ? base + c * 16 : (const char*)kZeros, to + T::kRopes + first * T::kRope);
        }
      }
    } else {
      constexpr int kCodes = kLatent / 16, kPer = 64 / kCodes;  // chunks of 16 codes per row, rows per load
#pragma unroll
      for (int i = 0; i < kLatentLoads; ++i) {
        const int row = (part * kLatentLoads + i) * kPer + lane / kCodes, c = lane % kCodes;
        const char* const base = row_of(lat, row);
        const uint8_t* const scale = row_of(sc, row);
        const bool in = c * 16 < P.C.latent;
        codes[i] = *(const u32x4*)(in ? base + c * 16 : (const char*)kZeros);
        scales[i] = in ? scale[c / 2] : 0;
      }
      if (P.C.rope > 0) {
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
          const int row = (part * kRopeLoads + i) * 8 + lane / 8, c = lane % 8;
          const char* const base = row_of(rop, row);
          ropes[i] = *(const u32x4*)(c * 8 < P.C.rope ? base + c * 16 : (const char*)kZeros);
        }
      }
    }
  }

  // 8 bits: from the registers to LDS, as 16-bit values (exact: 4 bits times a power of two).
  __device__ __forceinline__ void land(const AttendParams& P, lds_char* to, int part, int lane) {
    lane = (int)fresh(lane);
    if constexpr (kE4m3) {
      constexpr int kCodes = kLatent / 16, kPer = 64 / kCodes;
#pragma unroll
      for (int i = 0; i < kLatentLoads; ++i) {
        const int row = (part * kLatentLoads + i) * kPer + lane / kCodes, c = lane % kCodes;
        const float f = scale_value(scales[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(codes[i][2 * h + j], false);
            const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(codes[i][2 * h + j], true);
            v[4 * j] = f * a.x;
            v[4 * j + 1] = f * a.y;
            v[4 * j + 2] = f * b.x;
            v[4 * j + 3] = f * b.y;
          }
          *(__attribute__((address_space(3))) u32x4*)(to + row * T::kRow + ((2 * c + h) ^ T::latent_flip(row)) * 16) =
              pack_eight<kF>(v);
        }
      }
      if (P.C.rope > 0) {
#pragma unroll
        for (int i = 0; i < kRopeLoads; ++i) {
          const int row = (part * kRopeLoads + i) * 8 + lane / 8, c = lane % 8;
          *(__attribute__((address_space(3))) u32x4*)(to + T::kRopes + row * T::kRope + (c ^ T::rope_flip(row)) * 16) = ropes[i];
        }
      }
    }
  }
};

// A row's largest score may grow by this (in powers of two) before its sums are rescaled.
constexpr float kSlack = 8.0f;
constexpr float kLowest = -3.402823466e38f;

template <int kF, int kLatent, int kQ, bool kE4m3>
__global__ __launch_bounds__(64 * kAttendWaves, 1) void latent_attend_kernel(AttendParams P) {
  using T = Tile<kLatent>;
  constexpr int kSplit = kAttendWaves / kQ;  // waves that share a block of 16 rows, each with its own keys
  constexpr int kIter = kTileKeys * kSplit, kRows = 16 * kQ;
  constexpr int kSteps = kLatent / 32, kColumns = kLatent / 16;
  using L = Line<kRows, kIter>;
  // Every kQ waves have a ring of kQ tiles: four tiles in all.
  constexpr int kSumRow = kLatent + 4;  // floats per row of sums, off the banks' period
  constexpr int kTiles = kAttendWaves * T::kBytes, kSums = kAttendWaves * 16 * kSumRow * 4;
  __shared__ __attribute__((aligned(16))) char memory[kTiles > kSums ? kTiles : kSums];
  __shared__ float tops[kAttendWaves][16], totals[kAttendWaves][16];
  __shared__ __attribute__((aligned(16))) char room[128];

  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  const int q = wave % kQ, split = wave / kQ, g = lane / 16, n = lane % 16;
  Place from, to;
  int64_t all;
  const int workers = find_part<kRows, kIter>(P, room, from, to, all);
  const int w = blockIdx.x;
  if (tid == 0) P.pieces[4 * w + 2] = 0;
  if (w >= workers || all == 0) return;

  lds_char* const tiles = (lds_char*)memory + split * kQ * T::kBytes;
  const lds_char* key_at[4];  // chunk 4 k + g of row n, for k % 4
  const lds_char* rope_at[2];
  const lds_char* column_at[8];  // columns 16 c .. of rows 4 g .. , for c % 8
#pragma unroll
  for (int k = 0; k < 4; ++k) key_at[k] = tiles + n * T::kRow + ((4 * k + g) ^ T::latent_flip(n)) * 16;
#pragma unroll
  for (int k = 0; k < 2; ++k) rope_at[k] = tiles + T::kRopes + n * T::kRope + ((4 * k + g) ^ T::rope_flip(n)) * 16;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int row = 4 * g + n / 4;
    column_at[c] = tiles + row * T::kRow + ((2 * c + n % 4 / 2) ^ T::latent_flip(row)) * 16 + n % 2 * 8;
  }

  for (Place at = from; at.before(to);) {
    int start;
    const int tokens = L::tokens(P, at.s, start);
    if (tokens == 0) {
      at = Place{at.s + 1, 0, 0};
      continue;
    }
    const int keys = L::keys(P, at.s), blocks = L::blocks(P, tokens), every = L::tiles(keys);
    const bool ends = at.s < to.s || at.b < to.b;
    const int t1 = ends ? every : to.t;
    // The row of this lane's query, its token and how many keys it sees.
    const int rows = tokens * (int)P.heads.d, row = at.b * kRows + q * 16 + n;
    const bool live = row < rows;
    const int token = (int)P.heads(live ? row : 0), head = (live ? row : 0) - token * (int)P.heads.d;
    const int past = P.seq_lens[at.s] - tokens + 1;  // what token 0 sees
    const int reach = past + token;
    const int least = past + (int)P.heads(at.b * kRows + q * 16 < rows ? at.b * kRows + q * 16 : rows - 1);
    const int last_row = (at.b + 1) * kRows < rows ? (at.b + 1) * kRows - 1 : rows - 1;
    const int most = past + (int)P.heads(last_row);
    const int seen = most < 0 ? 0 : (most < keys ? most : keys);
    const int count = (t1 < L::tiles(seen) ? t1 : L::tiles(seen)) - at.t;  // tiles to go; may be negative

    u32x4 qf[kSteps], qx[2];
    {
      const char* const a = P.ql + (start + token) * P.ql_ts + head * P.ql_hs;
      const char* const b = P.qr + (start + token) * P.qr_ts + head * P.qr_hs;
      const int c = (int)fresh(g * 8);
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        qf[k] = *(const u32x4_any*)(live && k * 32 + c < P.C.latent ? a + (k * 32 + c) * 2 : (const char*)kZeros);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        qx[k] = *(const u32x4_any*)(live && k * 32 + c < P.C.rope ? b + (k * 32 + c) * 2 : (const char*)kZeros);
    }
    f32x4 O[kColumns];
#pragma unroll
    for (int c = 0; c < kColumns; ++c) O[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float top = kLowest, weight = 0.0f;

    const int first_key = at.t * kIter + split * kTileKeys;
    Loader<kF, kLatent, kQ, kE4m3> load;
    uint32_t masks[kQ];  // of the tiles under way, the next to be worked on first

    // Works on the tile in ring place `slot`, keys from `key` on.
    const auto work = [&](int slot, int key, uint32_t mask) {
      const int off = slot * T::kBytes;
      f32x4 S[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) S[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          S[i][k % 2] = mfma_16x16x32<kF>(lds_read16(key_at[k % 4] + off + i * 16 * T::kRow + k / 4 * 256), qf[k], S[i][k % 2]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          S[i][k] = mfma_16x16x32<kF>(lds_read16(rope_at[k] + off + i * 16 * T::kRope), qx[k], S[i][k]);
      interleave<2 * kSteps + 4>();
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (S[i / 4][0][i % 4] + S[i / 4][1][i % 4]) * P.scale;
      bool unsafe = false;
      if (mask != 0xFFFFFFFFu || key + kTileKeys > least) {
        // Rows that do not see a key have weight 0 for it, but 0 times NaN is NaN. A key with a
        // value that is not finite gives every row such a score.
        float worst = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) worst += 0.0f * x[i];
        unsafe = most != least && __ballot(worst != 0.0f) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = i / 4 * 16 + 4 * g + i % 4;
          if (!((mask >> k) & 1) || key + k >= reach) x[i] = -__builtin_huge_valf();
        }
      }
      float now = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) now = __builtin_fmaxf(now, x[i]);
      now = __builtin_fmaxf(now, __shfl_xor(now, 16));
      now = __builtin_fmaxf(now, __shfl_xor(now, 32));
      if (__ballot(now > top + kSlack) != 0) {
        const float next = __builtin_fmaxf(top, now), f = exp2_hw(top - next);
        top = next;
        weight *= f;
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
          O[c] *= f;
          if (c % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
      }
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_hw(x[i] - top);
        weight += p[i];
      }
      const u32x4 pf = pack_eight<kF>(p);
      if (unsafe) {
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
          const lds_char* const a = column_at[c % 8] + off + c / 8 * 256;
          const u32x2 u = finite_pairs<kF>(lds_read_columns(a)), v = finite_pairs<kF>(lds_read_columns(a + 16 * T::kRow));
          O[c] = mfma_16x16x32<kF>(u32x4{u[0], u[1], v[0], v[1]}, pf, O[c]);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
          const lds_char* const a = column_at[c % 8] + off + c / 8 * 256;
          const u32x2 u = lds_read_columns(a), v = lds_read_columns(a + 16 * T::kRow);
          O[c] = mfma_16x16x32<kF>(u32x4{u[0], u[1], v[0], v[1]}, pf, O[c]);
        }
        interleave_pairs<kColumns>();
      }
    };

    // Rotated parts that are never loaded are zeros; the last block's sums lay there.
    if (P.C.rope == 0) {
      static_assert(T::kBytes - T::kRopes == 16 * 64 * kAttendWaves, "a thread clears 16 bytes of each tile");
      for (int i = 0; i < kAttendWaves; ++i)
        ((u32x4*)(memory + i * T::kBytes + T::kRopes))[tid] = u32x4{0, 0, 0, 0};
      __syncthreads();
    }
    if (count > 0) {
      if constexpr (kE4m3) {
        load.find(P, at.s, first_key, keys, lane);
        load.issue(P, tiles, q, lane);
        for (int i = 0; i < count; ++i) {
          const int slot = i % kQ;
          const uint32_t mask = load.mask;
          // (The wave's own reads and writes; LDS serves a wave in order.)
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          load.land(P, tiles + slot * T::kBytes, q, lane);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          if (i + 1 < count) {
            load.find(P, at.s, first_key + (i + 1) * kIter, keys, lane);
            load.issue(P, tiles, q, lane);
          }
          if (kQ > 1) __syncthreads();
          work(slot, first_key + i * kIter, mask);
        }
      } else if constexpr (kQ == 1) {
        load.find(P, at.s, first_key, keys, lane);
        load.issue(P, tiles, q, lane);
        for (int i = 0; i < count; ++i) {
          const uint32_t mask = load.mask;
          if (i + 1 < count) load.find(P, at.s, first_key + (i + 1) * kIter, keys, lane);
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          work(0, first_key + i * kIter, mask);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          if (i + 1 < count) load.issue(P, tiles, q, lane);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kQ - 1; ++i) {
          if (i < count) {
            load.find(P, at.s, first_key + i * kIter, keys, lane);
            load.issue(P, tiles + i * T::kBytes, q, lane);
            masks[i] = load.mask;
          }
        }
        int slot = 0;
        for (int i = 0; i < count; ++i) {
          // This wave's part of tile i has arrived; after the barrier everyone's has, and
          // everyone is done with tile i - 1.
          if (i + kQ - 1 < count + 1)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kQ - 2) * Loader<kF, kLatent, kQ, kE4m3>::kLatentLoads) : "memory");
          else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          __syncthreads();
          const uint32_t mask = masks[0];
#pragma unroll
          for (int j = 0; j + 1 < kQ - 1; ++j) masks[j] = masks[j + 1];
          if (i + kQ - 1 < count) {
            load.find(P, at.s, first_key + (i + kQ - 1) * kIter, keys, lane);
            load.issue(P, tiles + (slot == 0 ? kQ - 1 : slot - 1) * T::kBytes, q, lane);
            masks[kQ - 2] = load.mask;
          }
          work(slot, first_key + i * kIter, mask);
          slot = slot + 1 == kQ ? 0 : slot + 1;
        }
      }
    }
    weight += __shfl_xor(weight, 16);
    weight += __shfl_xor(weight, 32);

    // The waves' sums of a row come together in LDS, and go out.
    if (g == 0) {
      tops[wave][n] = top;
      totals[wave][n] = weight;
    }
    __syncthreads();  // tiles are no longer read
    float high = tops[q][n];
#pragma unroll
    for (int i = 1; i < kSplit; ++i) high = __builtin_fmaxf(high, tops[i * kQ + q][n]);
    float f = exp2_hw(top - high), total = 0.0f;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) total = __builtin_fmaf(totals[i * kQ + q][n], exp2_hw(tops[i * kQ + q][n] - high), total);
    const bool whole = at.t == 0 && t1 == every;
    if (whole) f *= total == 0.0f ? 0.0f : 1.0f / total;
    float* const sums = (float*)memory;
#pragma unroll
    for (int c = 0; c < kColumns; ++c) *(f32x4*)(sums + (wave * 16 + n) * kSumRow + 16 * c + 4 * g) = f * O[c];
    const Partial part{kRows, P.C.latent};
    float* const mine = P.partial + part.floats() * (2 * w + (ends ? 0 : 1));
    if (!whole && split == 0 && g == 0) {
      mine[part.exponent() + q * 16 + n] = high;
      mine[part.weight() + q * 16 + n] = total;
    }
    __syncthreads();
    constexpr int kEights = kLatent / 8;
    for (int i = tid; i < kRows * kEights; i += 64 * kAttendWaves) {
      const int r = i / kEights, c = i % kEights * 8;
      if (c >= P.C.latent || at.b * kRows + r >= rows) continue;
      float v[8] = {};
#pragma unroll
      for (int k = 0; k < kSplit; ++k) {
        const float* const a = sums + ((k * kQ + r / 16) * 16 + r % 16) * kSumRow + c;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += a[j];
      }
      if (whole) {
        const int64_t to_row = (int64_t)start * P.heads.d + at.b * kRows + r;
        store_eight<kF>(P.out + (to_row * P.C.latent + c) * 2, v);
      } else {
        *(f32x4*)(mine + (int64_t)r * P.C.latent + c) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(mine + (int64_t)r * P.C.latent + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
    // The worker that begins a shared block says how many have a part of it.
    if (tid == 0 && at.t == 0 && !ends) {
      // Units up to the block's end: this worker's part ends to.t + kBlockUnits units into it.
      const int64_t end = all * (w + 1) / workers - (to.t + kBlockUnits) + every + kBlockUnits;
      const int64_t last = (end * workers + all - 1) / all;  // the first worker that begins at or past it
      P.pieces[4 * w] = at.s;
      P.pieces[4 * w + 1] = at.b;
      P.pieces[4 * w + 2] = (int)(last - w);
    }
    __syncthreads();
    at = at.b + 1 < blocks ? Place{at.s, at.b + 1, 0} : Place{at.s + 1, 0, 0};
  }
}

// Joins the parts of shared blocks: one wave per row.
template <int kF, int kRows>
__global__ __launch_bounds__(256) void latent_join_kernel(AttendParams P) {
  const int w = blockIdx.x, lane = threadIdx.x % 64;
  const int count = P.pieces[4 * w + 2];
  if (count == 0) return;
  const int s = P.pieces[4 * w], b = P.pieces[4 * w + 1];
  int start;
  const int tokens = Line<kRows, 1>::tokens(P, s, start);
  const int r = blockIdx.y * 4 + uniform(threadIdx.x / 64);
  if (b * kRows + r >= tokens * (int)P.heads.d) return;
  const Partial part{kRows, P.C.latent};
  const auto slot = [&](int i) { return P.partial + part.floats() * (2 * (w + i) + (i + 1 < count)); };
  float high = kLowest;
  for (int i = lane; i < count; i += 64) high = __builtin_fmaxf(high, slot(i)[part.exponent() + r]);
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) high = __builtin_fmaxf(high, __shfl_xor(high, m));
  const int c = lane * 8;
  const bool mine = c < P.C.latent;
  float total = 0.0f, v[8] = {};
  for (int base = 0; base < count; base += 64) {
    float f = 0.0f, l = 0.0f;
    if (base + lane < count) {
      const float* const a = slot(base + lane);
      f = exp2_hw(a[part.exponent() + r] - high);
      l = f * a[part.weight() + r];
    }
    total += lane_sum<64>(l);
    const int here = count - base < 64 ? count - base : 64;
    // Four parts' loads at a time.
    for (int i = 0; i < here; i += 4) {
      f32x4 lo[4], hi[4];
      float fs[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = i + k < here ? i + k : here - 1;
        fs[k] = i + k < here ? __shfl(f, at) : 0.0f;
        const f32x4* const a = (const f32x4*)(slot(base + at) + (int64_t)r * P.C.latent + (mine ? c : 0));
        lo[k] = a[0];
        hi[k] = a[1];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i + k >= here) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = __builtin_fmaf(fs[k], lo[k][j], v[j]);
          v[4 + j] = __builtin_fmaf(fs[k], hi[k][j], v[4 + j]);
        }
      }
    }
  }
  const float f = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= f;
  if (mine) store_eight<kF>(P.out + (((int64_t)start * P.heads.d + b * kRows + r) * P.C.latent + c) * 2, v);
}

template <int kF, int kLatent, int kQ, bool kE4m3>
void launch_attend(const AttendParams& P, hipStream_t st) {
  hipLaunchKernelGGL((latent_attend_kernel<kF, kLatent, kQ, kE4m3>), dim3(P.workers), dim3(64 * kAttendWaves), 0, st, P);
  hipLaunchKernelGGL((latent_join_kernel<kF, 16 * kQ>), dim3(P.workers, 4 * kQ), dim3(256), 0, st, P);
}

}  // namespace kdaconv

#endif  // KDACONV_LATENT_ATTENTION_DEVICE_H_
