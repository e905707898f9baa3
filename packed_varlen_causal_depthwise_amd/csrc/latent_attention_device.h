// Absorbed latent attention over the paged cache: the kernels.
//
// For a row (a head of a new token) with query (ql, qr) and the cached tokens t below its reach
//     s_t = scale (ql . c_t + qr . r_t),  out = sum_t softmax(s)_t c_t
// so a token's latent is key and value at once: it goes to LDS once and is read there twice.
//
// A workgroup of 8 waves holds kQ blocks of 16 rows and takes the keys in steps. For the scores
// a wave takes one block's products with 16 or 32 keys over all channels, for the sums all
// blocks' with its own 64 columns (of 512): between the two the weights go through LDS. So
// no wave holds more than 64 sums and 72 registers of queries, columns are read once, and two
// waves share each SIMD.
//
// What bounds it: with few rows memory. 256 sequences of 12 heads over a million keys of 512 + 64
// bf16 channels, 1.2 GB, take 240 us with the join (5.6 TB/s alone; plain reads reach 6.0), a step
// of 32 keys 2450 cycles, in which LDS takes its 36 KB at 1 KB in some 45 cycles. With 64 rows memory
// still: 24 chunks of 500 tokens in all, 8 heads, 70007 keys take 78 us, 330 TFLOP/s. Blocks of one
// sequence are at different keys at any one time, so keys come three times (272 MB read and 35 MB
// of sums written: 62 us at a copy's rate); LDS reads of 420 KB a step take some 18. With few keys
// latency: some 3000 cycles until a worker has found its part, 6000 more until the first keys are
// there.
//
// Products are taken transposed, S^T = K Q^T and O^T = C^T P^T: a lane then has one query, whose
// largest score and rescaling concern no other lane. The left operand C^T is delivered by
// LDS: ds_read_b64_tr_b16 hands 16 lanes the columns of 4 rows of 16.
#ifndef KDACONV_LATENT_ATTENTION_DEVICE_H_
#define KDACONV_LATENT_ATTENTION_DEVICE_H_

#include "attention_device.h"
#include "latent_attention.h"

namespace kdaconv {

// A place on the line of work: sequence, block of rows, tile of keys.
struct Place {
  int s, b, t;
  __device__ bool before(const Place& o) const { return s < o.s || (s == o.s && (b < o.b || (b == o.b && t < o.t))); }
};

template <int kRows, int kKeys>
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
  static __device__ __forceinline__ int keys(const AttendParams& P, int n) {
    return n < 0 ? 0 : (n > P.most_keys ? P.most_keys : n);
  }
  // (Rows are below 2^29 and keys up to 2^30.)
  static __device__ __forceinline__ int blocks(const AttendParams& P, int tokens) {
    return (tokens * (int)P.heads.d + kRows - 1) / kRows;
  }
  static __device__ __forceinline__ int tiles(const AttendParams& P, int keys) {
    const int steps = (int)((uint32_t)(keys + kKeys - 1) / kKeys);
    return (steps + (1 << P.shift) - 1) >> P.shift;
  }
};

// Equal parts of a line of `total` units: the first `rest` are one longer than the others.
struct Parts {
  int count, each, rest;
  __device__ __forceinline__ Parts(int total, int most) {
    count = total < most * kLeastUnits ? total / kLeastUnits : most;
    count = count < 1 ? 1 : count;
    each = (int)((uint32_t)total / (uint32_t)count);
    rest = total - each * count;
  }
  __device__ __forceinline__ int begin(int i) const { return each * i + (i < rest ? i : rest); }
};

// Sum of the lanes up to each, in the vector unit.
__device__ __forceinline__ int running_sum(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // 1, 2, 4 and 8 lanes down a row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // a row's last to the next, to rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return x;
}

// Finds this worker's part of the line. All threads of the workgroup call it; `room` is LDS of
// 96 bytes.
template <int kRows, int kKeys>
__device__ __forceinline__ Parts find_part(const AttendParams& P, char* room, Place& from, Place& to) {
  using L = Line<kRows, kKeys>;
  int* const sums = (int*)room;  // per wave, of the first sequences
  int* const rests = sums + kAttendWaves;  // of the others
  int* const found = rests + kAttendWaves;  // from, to
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  constexpr int kThreads = 64 * kAttendWaves;
  int per = 0;  // units of a block
  const auto units = [&](int s) {
    if (s >= P.seqs) return 0;
    int start;
    const int n = L::tokens(P, s, start);
    per = L::tiles(P, L::keys(P, P.seq_lens[s])) + kBlockUnits;
    return L::blocks(P, n) * per;
  };
  int u = units(tid), run = running_sum(u);
  if (lane == 63) sums[wave] = run;
  const bool many = P.seqs > kThreads;
  if (many) {
    const int mine = per;
    int rest = 0;
    for (int s = tid + kThreads; s < P.seqs; s += kThreads) rest += units(s);
    rest = running_sum(rest);
    if (lane == 63) rests[wave] = rest;
    per = mine;
  } else if (lane == 63) {
    rests[wave] = 0;
  }
  if (tid < 6) found[tid] = tid % 3 == 0 ? P.seqs : 0;
  __syncthreads();
  int first = 0, next = 0, total = 0;  // units before this thread's sequence, before the next thread 0's
#pragma unroll
  for (int i = 0; i < kAttendWaves; ++i) {
    if (i < wave) first += sums[i];
    next += sums[i];
    total += rests[i];
  }
  total += next;
  const Parts parts(total, P.workers);
  const int w = blockIdx.x, lo = parts.begin(w), hi = parts.begin(w + 1);
  for (int s = tid;;) {
    first += run - u;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int off = (e == 0 ? lo : hi) - first;
      if (off >= 0 && off < u) {
        const int b = (int)((uint32_t)off / (uint32_t)per), r = off - b * per;
        found[3 * e] = s;
        found[3 * e + 1] = b;
        found[3 * e + 2] = r > kBlockUnits ? r - kBlockUnits : 0;
      }
    }
    __syncthreads();
    s += kThreads;
    if (s - tid >= P.seqs || next > hi) break;
    u = units(s);
    run = running_sum(u);
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    first = next;
#pragma unroll
    for (int i = 0; i < kAttendWaves; ++i) {
      if (i < wave) first += sums[i];
      next += sums[i];
    }
  }
  from = Place{uniform(found[0]), uniform(found[1]), uniform(found[2])};
  to = Place{uniform(found[3]), uniform(found[4]), uniform(found[5])};
  if (w >= parts.count) to = from;
  return parts;
}

// LDS of a step's keys: their latents, then their rotated parts, rows of 16-byte chunks. Chunk
// c of row r lies at place c ^ f(r) of its row, with f such that neither 16 rows' chunk c (the
// scores' left operand) nor chunks 2 i, 2 i + 1 of rows 0 to 3 and 8 to 11, or 4 to 7 and 12 to 15
// (columns), share a bank.
template <int kLatent, int kKeys>
struct Tile {
  static constexpr int kRow = kLatent * 2, kRope = kRopeMax * 2;
  static constexpr int kRopes = kKeys * kRow;
  static constexpr int kBytes = kRopes + kKeys * kRope;
  static __device__ __forceinline__ int latent_flip(int row) {
    return ((row & 3) << 1) | ((row >> 3 & 1) << 3) | (row >> 2 & 1);
  }
  static __device__ __forceinline__ int rope_flip(int row) { return (row >> 1) & 7; }
};

// Where 64 keys lie: lane i has key i.
template <bool kE4m3>
struct Keys {
  int window = -1;  // page of number window_at + lane of sequence window_of
  int window_at = 0, window_of = -1;
  const char* lat;  // zeros where there is no key
  const char* rop;
  const uint8_t* sc;
  uint64_t mask;  // keys that are there

  // Finds the keys from `first` on. The lanes hold a window of the page table: loads return in
  // order, so an entry loaded for each step would wait for all steps under way.
  __device__ __forceinline__ void find(const AttendParams& P, int s, int first, int keys, int lane) {
    lane = (int)fresh(lane);
    const int end = first + 64 < keys ? first + 64 : keys;
    const int low = (int)P.C.page_size((uint32_t)first);
    if (window_of != s || low < window_at || (end > first && (int)P.C.page_size((uint32_t)(end - 1)) >= window_at + 64)) {
      window_of = s;
      window_at = low;
      window = low + lane < P.T.width ? P.T.table[s * P.T.stride + low + lane] : -1;
      // (Here and not at its use, which every step would wait for.)
      asm volatile("s_waitcnt vmcnt(0)" : "+v"(window));
    }
    const int key = first + lane;
    const uint32_t p = P.C.page_size((uint32_t)key);
    const int at = key - (int)(p * P.C.page_size.d);
    const int page = __shfl(window, (int)p - window_at);
    const bool ok = key < keys && page >= 0 && page < P.C.num_pages;
    mask = __ballot(ok);
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
};

// A step from memory to LDS, 16 bits straight, by kLoaders waves in turn: a load takes one row's
// latent of 512 channels or two of 256, or 8 rows' rotated parts.
template <int kLatent, int kKeys, int kLoaders>
struct Direct {
  using T = Tile<kLatent, kKeys>;
  static constexpr int kChunks = kLatent / 8, kPer = 64 / kChunks;  // chunks per row, rows per load
  static constexpr int kLatents = kKeys / kPer, kAll = kLatents + kKeys / 8;  // loads
  static constexpr int kTurns = (kAll + kLoaders - 1) / kLoaders;
  static constexpr int kLeast = kLatents / kLoaders;  // of every wave, whatever the sizes

  // Turns `begin` to `end` of this wave. `base`: the lane that has the step's first key.
  static __device__ __forceinline__ void issue(const AttendParams& P, const Keys<false>& K, int base, lds_char* to,
                                               int loader, int lane, int begin, int end) {
    // Flips reach 16 chunks. Where latents end at a multiple of them a lane is past the end by
    // its number alone: it reads the first chunks (queries are zero there, and no sum is taken).
    const bool even = P.C.latent % 128 == 0;
    const int c = lane % kChunks;
    const uint32_t at = (c * 8 < P.C.latent ? c : c % 16) * 16;
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      if (j < begin || j >= end) continue;
      const int i = loader + j * kLoaders;
      if (i < kLatents) {
        const int first = i * kPer, row = first + (kPer == 1 ? 0 : lane / kChunks);
        const uint32_t flip = T::latent_flip(row);
        if (even) {
          if constexpr (kPer == 1)
            to_lds16(K.row_uniform(K.lat, base + first), at ^ (flip * 16), to + first * T::kRow);
          else
            to_lds16(K.row_of(K.lat, base + row) + (at ^ (flip * 16)), to + first * T::kRow);
        } else {
          const char* const from = K.row_of(K.lat, base + row);
          const int chunk = c ^ flip;
          to_lds16(chunk * 8 < P.C.latent ? from + chunk * 16 : (const char*)kZeros, to + first * T::kRow);
        }
      } else if (i < kAll && P.C.rope > 0) {
        const int first = (i - kLatents) * 8, row = first + lane / 8, chunk = lane % 8 ^ T::rope_flip(row);
        const char* const from = K.row_of(K.rop, base + row);
        to_lds16(chunk * 8 < P.C.rope ? from + chunk * 16 : (const char*)kZeros, to + T::kRopes + first * T::kRope);
      }
    }
  }
};

// 8 bits by way of registers, where they become 16-bit values (exactly, within fp16's range: 4
// bits times a power of two). A wave takes 8 rows, of each 8 lanes every eighth chunk of 16 codes:
// a row's addresses are found once, and the chunks' flips are the same for all of a lane's.
template <int kF, int kLatent, int kKeys>
struct Staged {
  using T = Tile<kLatent, kKeys>;
  static constexpr int kRows = 8, kLoads = kLatent / 128;
  // A step's registers: codes, the rotated part, scales.
  static constexpr int kRegisters = kLoads + 2;
  static_assert(kLoads <= 4);

  static __device__ __forceinline__ void issue(const AttendParams& P, const Keys<true>& K, int first, int wave, int lane,
                                               u32x4* set) {
    const uint32_t at = fresh(lane), c = at % 8, row = first + wave * kRows + at / 8;
    const auto codes = (Global<char>)K.row_of(K.lat, row), rope = (Global<char>)K.row_of(K.rop, row);
    const auto scales = (Global<uint8_t>)K.row_of(K.sc, row);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // (Past the end the first chunk: queries are zero there, and no sum is taken.)
      const uint32_t chunk = (c + 8 * i) * 16 < (uint32_t)P.C.latent ? c + 8 * i : 0;
      set[i] = *(Global<u32x4>)(codes + chunk * 16);
    }
    // Chunk c + 8 i has scale c / 2 + 4 i: that byte of word i.
    if (P.C.latent == kLatent) {
      typedef uint32_t words __attribute__((ext_vector_type(kLoads), aligned(1)));
      const words w = *(Global<words>)scales;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) set[kLoads + 1][i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t chunk = (c + 8 * i) * 16 < (uint32_t)P.C.latent ? c + 8 * i : 0;
        set[kLoads + 1][i] = scales[chunk / 2] << (c / 2 * 8);
      }
    }
    const auto zeros = (Global<char>)(const char*)kZeros;
    set[kLoads] = *(Global<u32x4>)(c * 8 < (uint32_t)P.C.rope ? rope + c * 16 : zeros);
  }

  static __device__ __forceinline__ void land(lds_char* to, int wave, int lane, const u32x4* set) {
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    const uint32_t at = fresh(lane), c = at % 8, row = wave * kRows + at / 8;
    const uint32_t even = row * T::kRow + ((2 * c) ^ T::latent_flip(row)) * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const float f = scale_value(set[kLoads + 1][i] >> (c / 2 * 8) & 255);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[2 * j] = scaled_pair<kF, false>(set[i][2 * h + j], f);
          v[2 * j + 1] = scaled_pair<kF, true>(set[i][2 * h + j], f);
        }
        *(lds_u32x4*)(to + (even ^ (h * 16)) + i * 256) = v;
      }
    }
    *(lds_u32x4*)(to + T::kRopes + row * T::kRope + (c ^ T::rope_flip(row)) * 16) = set[kLoads];
  }
};

template <int kF, int kLatent, int kQ, bool kE4m3>
__global__ __launch_bounds__(64 * kAttendWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void latent_attend_kernel(AttendParams P) {
  constexpr int kKeys = step_keys(kQ), kRing = ring_steps(kQ), kRows = 16 * kQ;
  using T = Tile<kLatent, kKeys>;
  using L = Line<kRows, kKeys>;
  constexpr int kSteps = kLatent / 32;  // products per score, beside two for the rotated part
  constexpr int kColumns = kLatent / 16 / kAttendWaves;  // blocks of 16 columns per wave
  // For the scores, wave w takes row block w % kQ and key blocks of 16 from kPart (w / kQ) on.
  constexpr int kBlocks = kKeys / 16, kPart = kQ * kBlocks > kAttendWaves ? kQ * kBlocks / kAttendWaves : 1;
  // Weights: rows of kKeys 16-bit values, chunks flipped as rotated parts are.
  constexpr int kWeightRow = kKeys * 2, kFlips = kKeys / 8;
  __shared__ __attribute__((aligned(1024))) char memory[kRing * T::kBytes];
  static_assert(T::kBytes % 1024 == 0 && T::kRow % 256 == 0 && kColumns <= 4);
  __shared__ __attribute__((aligned(16))) char weights[kRows * kWeightRow];
  __shared__ __attribute__((aligned(16))) float tops[kRows][kBlocks];  // a step's largest scores
  __shared__ __attribute__((aligned(16))) char room[96];
  __shared__ uint64_t masks[4];  // of the keys of steps under way
  __shared__ __attribute__((aligned(16))) int bad[kLatent];  // a channel's first key that is not finite, of those made 0

  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  const int g = lane / 16, n = lane % 16;
  const int q = wave % kQ, kb = wave / kQ * kPart;
  const bool scores = kb < kBlocks;  // this wave takes part in them
  // Where some waves do not, they load (8 bits: four of them, with equal shares).
  constexpr int kIdle = kAttendWaves - kQ * kBlocks / kPart;
  constexpr int kLoaders = kIdle == 0 ? kAttendWaves : kE4m3 ? 4 : kIdle;
  const int loader = wave - (kAttendWaves - kLoaders);
  // Of 8-bit keys kSets steps are under way to registers, of waves that hold no queries where
  // there are such.
  using Load = Staged<kF, kLatent, kKeys>;
  static_assert(!kE4m3 || kKeys == kLoaders * Load::kRows);
  constexpr int kSets = kKeys == 64 ? 1 : 3, kSetsHold = kE4m3 ? kSets * Load::kRegisters : 0;
  constexpr int kHold = kIdle > 0 ? (kSetsHold > kSteps + 2 ? kSetsHold : kSteps + 2) : kSteps + 2 + kSetsHold;
  Place from, to;
  const Parts parts = find_part<kRows, kKeys>(P, room, from, to);
  const int w = blockIdx.x;
  if (tid < 2) P.shared[2 * w + tid].count = 0;
  if (!from.before(to)) return;

  const auto flip_weight = [](int row) { return kFlips == 8 ? (row >> 1) & 7 : (row >> 2) & 3; };
  lds_char* const tiles = (lds_char*)memory;
  // (A flip and a chunk's number are joined by xor, and tiles begin at multiples of 1024 bytes: so
  // chunk 4 k + g of a row is at (place of chunk g) ^ 64 k, and block c of columns at (place of
  // the wave's first) ^ 32 c.)
  const uint32_t key_at = (16 * kb + n) * T::kRow + (g ^ T::latent_flip(n)) * 16;
  const uint32_t rope_at = T::kRopes + (16 * kb + n) * T::kRope + (g ^ T::rope_flip(n)) * 16;
  // Columns: rows 8 g + n / 4 (the step's first 4 of 8) and 4 more, this wave's first block.
  uint32_t column_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * g + 4 * i + n / 4;
    column_at[i] = row * T::kRow + ((2 * wave * kColumns + n % 4 / 2) ^ T::latent_flip(row)) * 16 + n % 2 * 8;
  }
  const auto flipped = [&](uint32_t at, uint32_t by) { return tiles + (at ^ by); };

  // Rotated parts that are never loaded are zeros.
  if (P.C.rope == 0) {
    for (int r = 0; r < kRing; ++r)
      for (int i = tid; i < kKeys * 8; i += 64 * kAttendWaves)
        *(u32x4*)(memory + r * T::kBytes + T::kRopes + i * 16) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }

  Keys<kE4m3> find;
  for (Place at = from; at.before(to);) {
    int start;
    const int tokens = L::tokens(P, at.s, start);
    if (tokens == 0) {
      at = Place{at.s + 1, 0, 0};
      continue;
    }
    const int length = P.seq_lens[at.s];
    const int keys = L::keys(P, length), blocks = L::blocks(P, tokens), every = L::tiles(P, keys);
    const bool ends = at.s < to.s || at.b < to.b;
    const int t1 = ends ? every : to.t;
    // The row of this lane's query, its token and how many keys it sees.
    const int rows = tokens * (int)P.heads.d, row = at.b * kRows + q * 16 + n;
    const bool live = row < rows;
    const int token = (int)P.heads(live ? row : 0), head = (live ? row : 0) - token * (int)P.heads.d;
    const int past = length - tokens + 1;  // what token 0 sees
    const int reach = past + token;
    const int last_row = (at.b + 1) * kRows < rows ? (at.b + 1) * kRows - 1 : rows - 1;
    const int least = past + (int)P.heads(at.b * kRows), most = past + (int)P.heads(last_row);
    const int seen = most < 0 ? 0 : (most < keys ? most : keys);
    const bool differ = most != least;
    static_assert(kLatent <= 64 * kAttendWaves);
    if (differ && tid < kLatent) bad[tid] = INT32_MAX;
    // Steps to go; may be negative.
    const int begin = at.t << P.shift, last = (seen + kKeys - 1) / kKeys;
    const int count = ((t1 << P.shift) < last ? t1 << P.shift : last) - begin;
    const int first_key = begin * kKeys;

    u32x4 held[kHold];  // queries: chunks of 32 channels, then two of the rotated part
    if (scores) {
      const char* const a = P.ql + (start + token) * P.ql_ts + head * P.ql_hs;
      const char* const b = P.qr + (start + token) * P.qr_ts + head * P.qr_hs;
      const int c = (int)fresh(g * 8);
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        held[k] = *(Global<u32x4_any>)(live && k * 32 + c < P.C.latent ? a + (k * 32 + c) * 2 : (const char*)kZeros);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        held[kSteps + k] = *(Global<u32x4_any>)(live && k * 32 + c < P.C.rope ? b + (k * 32 + c) * 2 : (const char*)kZeros);
      // (They arrive here. Else every step would wait for them, and for the steps under way.)
#pragma unroll
      for (int k = 0; k < kSteps + 2; ++k) asm volatile("" : "+v"(held[k]));
    }
    u32x4* const set = held + (kIdle > 0 ? 0 : kSteps + 2);
    f32x4 O[kColumns][kQ];
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
#pragma unroll
      for (int i = 0; i < kQ; ++i) O[c][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float top[kQ];  // of rows 16 i + n, the same in every wave
#pragma unroll
    for (int i = 0; i < kQ; ++i) top[i] = kLowest;
    float my_top = kLowest, weight = 0.0f;  // of this lane's query: row q * 16 + n

    constexpr int kAll = (kSteps + 2) * kPart, kBatch = kQ == 4 ? 3 : kE4m3 ? 4 : 6, kBatches = (kAll + kBatch - 1) / kBatch;
    // One step, in ring place `slot`; everyone's share of it has arrived.
    // `send(j)`, for j below kBatches, is called along the scores.
    const auto work = [&](int step, int slot, auto send) {
      const int off = slot * T::kBytes, key = first_key + step * kKeys;
      const uint64_t mask = masks[step & 3];
      float x[kPart][4], sum;
      const auto weigh = [&]() {
        sum = 0.0f;
#pragma unroll
        for (int b = 0; b < kPart; ++b) {
          const f32x2 lo = {exp2_hw(x[b][0] - my_top), exp2_hw(x[b][1] - my_top)};
          const f32x2 hi = {exp2_hw(x[b][2] - my_top), exp2_hw(x[b][3] - my_top)};
          const int r = q * 16 + n, chunk = (kb + b) * 2 + g / 2;
          char* const p = weights + r * kWeightRow + (chunk ^ flip_weight(r)) * 16 + g % 2 * 8;
          Pair<kF>::store(p, lo);
          Pair<kF>::store(p + 4, hi);
          sum += (lo.x + lo.y) + (hi.x + hi.y);
        }
      };
      if (scores) {
        constexpr int kChains = kPart == 1 ? 2 : 1;  // (products that follow one another wait)
        f32x4 S[kPart][kChains];
#pragma unroll
        for (int b = 0; b < kPart; ++b)
          for (int j = 0; j < kChains; ++j) S[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // Operands are read a batch ahead of their products. (Left alone the compiler reads one,
        // waits for it and uses it.)
        const auto operand = [&](int i) {
          const int k = i / kPart, b = i % kPart;
          return k < kSteps ? lds_read16(flipped(key_at + off, k % 4 * 64) + b * 16 * T::kRow + k / 4 * 256)
                            : lds_read16(flipped(rope_at + off, (k - kSteps) * 64) + b * 16 * T::kRope);
        };
        u32x4 a[2][kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) a[0][i] = operand(i);
#pragma unroll
        for (int j = 0; j < kAll; j += kBatch) {
          send(j / kBatch);
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (j + kBatch + i < kAll) a[(j / kBatch + 1) % 2][i] = operand(j + kBatch + i);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (j + i >= kAll) break;
            const int k = (j + i) / kPart, b = (j + i) % kPart;
            S[b][k % kChains] = mfma_16x16x32<kF>(a[j / kBatch % 2][i], held[k], S[b][k % kChains]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        float now = -__builtin_huge_valf();
#pragma unroll
        for (int b = 0; b < kPart; ++b) {
          float high = -__builtin_huge_valf();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[b][i] = (kChains == 1 ? S[b][0][i] : S[b][0][i] + S[b][kChains - 1][i]) * P.scale;
            const int k = (kb + b) * 16 + 4 * g + i;
            if (mask != ~0ull >> (64 - kKeys) || key + kKeys > least)
              x[b][i] = ((mask >> k) & 1) && key + k < reach ? x[b][i] : -__builtin_huge_valf();
            high = __builtin_fmaxf(high, x[b][i]);
          }
          high = __builtin_fmaxf(high, __shfl_xor(high, 16));
          high = __builtin_fmaxf(high, __shfl_xor(high, 32));
          if (g == 0) tops[q * 16 + n][kb + b] = high;
          now = __builtin_fmaxf(now, high);
        }
        weigh();
      }
      lds_barrier();
      // The step's largest scores: all waves see the same and decide alike.
      float now[kQ];
      bool grows = false;
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const float* const a = tops[i * 16 + n];
        now[i] = __builtin_fmaxf(a[0], a[1]);
        if (kBlocks == 4) now[i] = __builtin_fmaxf(now[i], __builtin_fmaxf(a[2 % kBlocks], a[3 % kBlocks]));
        grows |= now[i] > top[i] + kSlack;
      }
      if (__ballot(grows) != 0) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const float next = __builtin_fmaxf(top[i], now[i]), f = exp2_hw(top[i] - next);
          top[i] = next;
#pragma unroll
          for (int c = 0; c < kColumns; ++c) O[c][i] *= f;
        }
        if (scores) {
          float next = my_top;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) next = __builtin_fmaxf(next, tops[q * 16 + n][b]);
          weight *= exp2_hw(my_top - next);
          my_top = next;
          weigh();
        }
        lds_barrier();
      }
      if (scores) weight += sum;
      // Rows that do not see a key have weight 0 for it, but 0 times NaN is NaN: where rows differ
      // in what they see, values that are not finite become zeros. The rows that see one have a
      // score that is not finite; if that is -inf their weight is 0 too, and they get their NaN at
      // the end. (What no row sees is not loaded.)
      if (differ && key + kKeys > least) {
        for (int i = (int)fresh(tid); i < T::kRopes / 16; i += 64 * kAttendWaves) {
          u32x4* const a = (u32x4*)(memory + off + i * 16);
          const u32x4 had = *a, has = finite_pairs<kF>(had);
          uint32_t change = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) change |= had[j] ^ has[j];
          if (change != 0) {
            *a = has;
            const int r = i / (kLatent / 8), c = (i % (kLatent / 8) ^ T::latent_flip(r)) * 8;
            for (int j = 0; j < 8; ++j)
              if (((had[j / 2] ^ has[j / 2]) >> (j % 2 * 16)) & 0xFFFF) atomicMin(&bad[c + j], key + r);
          }
        }
        lds_barrier();
      }
#pragma unroll
      for (int k = 0; k < kKeys / 32; ++k) {
        u32x4 p[kQ];
        u32x2 u[kColumns], v[kColumns];
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int r = i * 16 + n;
          p[i] = *(const u32x4*)(weights + r * kWeightRow + ((4 * k + g) ^ flip_weight(r)) * 16);
        }
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
          u[c] = lds_read_columns(flipped(column_at[0] + off, c * 32) + k * 32 * T::kRow);
          v[c] = lds_read_columns(flipped(column_at[1] + off, c * 32) + k * 32 * T::kRow);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < kColumns; ++c)
#pragma unroll
          for (int i = 0; i < kQ; ++i)
            O[c][i] = mfma_16x16x32<kF>(u32x4{u[c][0], u[c][1], v[c][0], v[c][1]}, p[i], O[c][i]);
      }
    };

    // Keys past the part's end, which are another worker's, and past what any row sees are loaded
    // as zeros: the latter have weight 0, but their values may be NaN.
    const int64_t part_end = (int64_t)first_key + (int64_t)count * kKeys;
    const int there = part_end < seen ? (int)part_end : seen;
    const auto find_step = [&](int step) {
      constexpr int kTimes = 64 / kKeys;  // steps that a search serves
      const int base = step % kTimes * kKeys;
      if (base == 0) find.find(P, at.s, first_key + step * kKeys, there, lane);
      if (loader == 0 && lane == 0) masks[step & 3] = find.mask << (64 - kKeys - base) >> (64 - kKeys);
      return base;
    };
    if (count > 0) {
      if constexpr (kE4m3) {
        // kSets steps are under way to registers; the next goes to LDS beside the present one.
        for (int base = -kSets; base < count; base += kSets) {
#pragma unroll
          for (int j = 0; j < kSets; ++j) {
            const int i = base + j;
            if (i >= count) break;
            if (i >= 0) lds_barrier();  // step i is in LDS, and everyone is done with step i - 1
            if (loader >= 0) {
              Load::issue(P, find, find_step(i + kSets), loader, lane, set + j * Load::kRegisters);
              if (kSets > 1 && i >= -1) 
                Load::land(tiles + ((i + 1) & 1) * T::kBytes, loader, lane, set + (j + 1) % kSets * Load::kRegisters);
            }
            if (i >= 0) work(i, i & 1, [](int) {});
            if (kSets == 1 && loader >= 0) Load::land(tiles + ((i + 1) & 1) * T::kBytes, loader, lane, set);
          }
        }
      } else {
        using D = Direct<kLatent, kKeys, kLoaders>;
        for (int i = 1 - kRing; i < count; ++i) {
          if (i >= 0) {
            // This wave's share of step i has arrived; after the barrier everyone's has, and
            // everyone is done with step i - 1, whose place is free.
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kRing - 2) * D::kLeast) : "memory");
            lds_barrier();
          }
          const int ahead = i + kRing - 1;
          lds_char* const to = tiles + (ahead & (kRing - 1)) * T::kBytes;
          if constexpr (kIdle > 0) {
            if (loader >= 0) D::issue(P, find, find_step(ahead), to, loader, (int)fresh(lane), 0, D::kTurns);
            if (i >= 0) work(i, i & (kRing - 1), [](int) {});
          } else {
            // A wave that sends faster than the loads are taken (1 KB in some 45 cycles of a CU)
            // stands: waves that have scores to do send along them.
            const int base = find_step(ahead), anew = (int)fresh(lane);
            const auto send = [&](int batch) {
              D::issue(P, find, base, to, loader, anew, (batch * D::kTurns + kBatches - 1) / kBatches,
                       ((batch + 1) * D::kTurns + kBatches - 1) / kBatches);
            };
            if (i >= 0)
              work(i, i & (kRing - 1), send);
            else
              D::issue(P, find, base, to, loader, anew, 0, D::kTurns);
          }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
    }

    // Each row's weight: this wave's lanes of it, then the waves that share it.
    weight += __shfl_xor(weight, 16);
    weight += __shfl_xor(weight, 32);
    __syncthreads();  // everyone has read the last step's largest scores
    if (scores && g == 0) tops[q * 16 + n][wave / kQ] = weight;
    __syncthreads();
    constexpr int kSums = kBlocks / kPart;
    const bool whole = at.t == 0 && t1 == every;
    const Partial part{kRows, P.C.latent};
    float* const mine = P.partial + part.floats() * (2 * w + (ends ? 0 : 1));
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int r = i * 16 + (kQ == 4 ? (int)fresh(n) : n);
      float total = tops[r][0];
#pragma unroll
      for (int j = 1; j < kSums; ++j) total += tops[r][j];
      if (!whole && wave == 0 && g == 0) {
        mine[part.exponent() + r] = top[i];
        mine[part.weight() + r] = total;
      }
      const float f = total == 0.0f ? 0.0f : 1.0f / total;
      if (at.b * kRows + r < rows) {
        const int sees = differ ? past + (int)P.heads(at.b * kRows + r) : 0;
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
          const int column = (wave * kColumns + c) * 16 + 4 * (kQ == 4 ? (int)fresh(g) : g);
          if (column >= P.C.latent) break;
          if (differ) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (bad[column + j] < sees) O[c][i][j] = __builtin_nanf("");
          }
          if (whole) {
            const f32x4 v = f * O[c][i];
            char* const o = P.out + (((int64_t)start * P.heads.d + at.b * kRows + r) * P.C.latent + column) * 2;
            Pair<kF>::store(o, f32x2{v[0], v[1]});
            Pair<kF>::store(o + 4, f32x2{v[2], v[3]});
          } else {
            *(f32x4*)(mine + (int64_t)r * P.C.latent + column) = O[c][i];
          }
        }
      }
    }
    // Who else has a part of this block: the last worker to begin at or before its first key (the
    // line's units count kBlockUnits before it) and those that begin after it, before its end.
    if (wave == 0 && !whole) {
      const int zero = at.t > 0 ? parts.begin(w) - at.t : parts.begin(w + 1) - to.t, end = zero + every;
      int before = 0, all = 0;
      for (int i = lane; __ballot(i < parts.count) != 0; i += 64) {
        const int at_unit = parts.begin(i);
        before += __builtin_popcountll(__ballot(i < parts.count && at_unit <= zero));
        all += __builtin_popcountll(__ballot(i < parts.count && at_unit < end));
      }
      // (Offsets that give rows to several sequences may wrap the line: still, all stays in range.)
      const int first = before > 0 ? before - 1 : 0;
      if (lane == 0) P.shared[2 * w + (ends ? 0 : 1)] = Shared{first, all > first ? all - first : 0, at.s, at.b};
    }
    __syncthreads();
    at = at.b + 1 < blocks ? Place{at.s, at.b + 1, 0} : Place{at.s + 1, 0, 0};
  }
}

// Joins the parts of shared blocks. Each worker that has a part joins its share of the block's
// rows and columns, 8 columns of a row at a time by as many lanes as take kJoinParts parts each.
// Its 7 us are a launch and three loads that follow one another; a last worker that joined alone
// would read one sequence's 167 parts, 5.5 MB, through one CU.
constexpr int kJoinThreads = 512, kJoinParts = 8;

template <int kF, int kRows>
__global__ __launch_bounds__(kJoinThreads) void latent_join_kernel(AttendParams P) {
  // The block that this worker's part begins inside, or the one that it ends inside.
  const int x = blockIdx.x, tid = threadIdx.x;
  const Partial part{kRows, P.C.latent};
  const Shared share = P.shared[2 * x + blockIdx.y];
  const int count = uniform(share.count), w = uniform(share.first);
  if (count == 0 || x < w || x - w >= count) return;
  int start;
  const int tokens = Line<kRows, 1>::tokens(P, uniform(share.s), start);
  int rows = tokens * (int)P.heads.d - uniform(share.b) * kRows;
  rows = rows < kRows ? rows : kRows;
  const int chunks = P.C.latent / 8, all = rows * chunks;
  const int from = (int)((uint32_t)(all * (x - w)) / (uint32_t)count), to = (int)((uint32_t)(all * (x - w + 1)) / (uint32_t)count);
  char* const out = P.out + ((int64_t)start * P.heads.d + uniform(share.b) * kRows) * P.C.latent * 2;
  const auto slot = [&](int i) { return P.partial + part.floats() * (2 * (w + i) + (i + 1 < count)); };
  int lanes = 1, log = 0;  // (at most 32: there are 256 workers)
  while (lanes * kJoinParts < count) lanes *= 2, ++log;
  const int turn = tid & (lanes - 1);
  for (int base = from; base < to; base += kJoinThreads >> log) {
    const int i = base + (tid >> log);
    const bool mine = i < to;
    const int r = (int)((uint32_t)(mine ? i : from) / (uint32_t)chunks), c = (mine ? i : from) - r * chunks;
    float e[kJoinParts], l[kJoinParts], high = kLowest, total = 0.0f;
    f32x4 a[kJoinParts][2], v[2] = {};
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k) {
      if (k * lanes >= count) break;
      const int number = turn + k * lanes;
      const float* const p = slot(number < count ? number : 0);
      e[k] = number < count ? p[part.exponent() + r] : kLowest;
      l[k] = p[part.weight() + r];
      const f32x4* const q = (const f32x4*)(p + (int64_t)r * P.C.latent + c * 8);
      a[k][0] = q[0];
      a[k][1] = q[1];
    }
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k)
      if (k * lanes < count) high = __builtin_fmaxf(high, e[k]);
    for (int m = lanes / 2; m > 0; m >>= 1) high = __builtin_fmaxf(high, __shfl_xor(high, m));
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k) {
      if (turn + k * lanes >= count) break;
      const float f = exp2_hw(e[k] - high);
      total = __builtin_fmaf(f, l[k], total);
      v[0] += f * a[k][0];
      v[1] += f * a[k][1];
    }
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j / 4][j % 4];
    for (int m = lanes / 2; m > 0; m >>= 1) {
      total += __shfl_xor(total, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += __shfl_xor(o[j], m);
    }
    const float f = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] *= f;
    if (mine && turn == 0) store_eight<kF>(out + ((int64_t)r * chunks + c) * 16, o);
  }
}

template <int kF, int kLatent, int kQ, bool kE4m3>
void launch_attend(const AttendParams& P, hipStream_t st) {
  hipLaunchKernelGGL((latent_attend_kernel<kF, kLatent, kQ, kE4m3>), dim3(P.workers), dim3(64 * kAttendWaves), 0, st, P);
  hipLaunchKernelGGL((latent_join_kernel<kF, 16 * kQ>), dim3(P.workers, 2), dim3(kJoinThreads), 0, st, P);
}

}  // namespace kdaconv

#endif  // KDACONV_LATENT_ATTENTION_DEVICE_H_
