// The gated delta rule in chunks of 32 tokens: the prefill.
//
// Mathematics. Inside a chunk let G_t be the running sum of the log decays (per key
// channel), k^ = k / |k| and n_t = |k_t| (or the normalised key and 1). With the state S at
// the chunk's start,
//     L_ti = b_t n_t n_i sum_c k^_tc k^_ic e^(G_tc - G_ic)   for i < t, else 0
//     T = diag(n) (I + L)^-1 diag(b)
//     U = T (V - diag(n) (K^ e^G) S)                         the updates, times n
//     O = scale |q| ((Q^ e^G) S + A U),  A_ti = sum_c q^_tc k^_ic e^(G_tc - G_ic), i <= t
//     S <- diag(e^G_end) S + (K^ e^(G_end - G))^T U
// so a chunk costs matrix products and one 32 x 32 triangular inverse instead of 32 steps.
// T and A do not depend on S.
//
// A long sequence is cut into segments. Over a segment S_end = M S_start + B: the scan of
// a segment from zero gives B, the scan of the identity without values gives M, and the
// starts follow by S_(j+1) = M_j S_j + B_j. Then all segments run side by side. (In one
// piece a sequence of 16384 tokens, 12 heads, would keep 12 CUs busy for 512 chunks of 4 us.)
//
// Kernels:
//   prepare   (chunk, head)             all that does not depend on S, into a slot
//   scan      (segment, head)           B and M, only for segments that others follow
//   join      (sequence, head, columns) the starts of the segments from the third on
//   scan      (segment, head)           outputs and the final state
// A chunk's gates, norms and exponentials are worked out once, by prepare, and handed over
// as matrix operands (60 KB per chunk and head of 128): the scans were bound by that vector
// work when they repeated it (5 us per chunk, 0.5 TB/s). One sequence of 16384 tokens, 12
// heads of 128, bf16 now takes 147 us in prepare, 113 for the transitions, 27 for the join
// and 99 for the outputs. Its tensors alone, 252 MB, are 50 us; the operands' way through
// memory, 1.1 GB of reads and writes more, and the chain from chunk to chunk are the rest.
//
// Numbers. Matrix products run on the FP16 matrix instructions with every operand split
// into a pair of FP16 values (22 bits) and three products: hi hi + hi lo + lo hi, summed
// in FP32. (One FP32 instruction costs as much as 16 FP16 ones of the same size; pairs of
// bfloat16 would keep 16 bits, which left the FP32 state 4e-6 off.) FP16's range holds
// because vectors have unit length, decays are at most 1, and a column's S and U share a
// power-of-two factor that follows the larger of them (U alone where a chunk empties S), while
// X = V - n Y may have one more of its own: with steps near 0 U is far below X, and pairs at X's
// scale would keep nothing of it. So errors are about 2^-22 of the largest value of a column in a
// chunk. T and A come from FP64
// and FP32 matrix instructions: their decays e^(G_t - G_i) are products of factors far
// outside FP16.
#ifndef KDACONV_DELTA_RULE_CHUNK_H_
#define KDACONV_DELTA_RULE_CHUNK_H_

#include "delta_rule_device.h"

namespace kdaconv {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32q __attribute__((ext_vector_type(4)));

constexpr float kVec = 16.0f;  // factor on stored unit vectors (their entries are small)
constexpr float kFaded = 0x1p-4f;  // a chunk whose decays are all below this empties the state

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// 16 bytes per lane from memory to LDS, at the wave's place + 16 times the lane's number.
// kLast: the memory is not read again.
template <bool kLast>
__device__ __forceinline__ void to_lds(const char* from, char* wave_to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)wave_to, 16, 0, kLast ? 2 : 0);
}

// x as an FP16 pair: hi rounded, lo the rounded rest.
struct HalfPair {
  f16x2 hi, lo;
};

// `one` is 1 in a register the compiler does not know: x one - hi then is one mixed-format
// fused multiply-add on the packed hi, where x - hi takes a conversion and a subtraction.
__device__ __forceinline__ HalfPair split2(f32x2 x, float one) {
  HalfPair p;
  p.hi = __builtin_convertvector(x, f16x2);
  p.lo = __builtin_convertvector(f32x2{__builtin_fmaf(x.x, one, -(float)p.hi.x),
                                      __builtin_fmaf(x.y, one, -(float)p.hi.y)}, f16x2);
  return p;
}

// Eight values (two tiles' four rows of one column) as matrix operands.
struct Operand {
  f16x8 hi, lo;
};

__device__ __forceinline__ Operand split8(f32x4 a, f32x4 b, float one) {
  Operand o;
  const HalfPair p0 = split2(f32x2{a[0], a[1]}, one), p1 = split2(f32x2{a[2], a[3]}, one);
  const HalfPair p2 = split2(f32x2{b[0], b[1]}, one), p3 = split2(f32x2{b[2], b[3]}, one);
  o.hi = f16x8{p0.hi.x, p0.hi.y, p1.hi.x, p1.hi.y, p2.hi.x, p2.hi.y, p3.hi.x, p3.hi.y};
  o.lo = f16x8{p0.lo.x, p0.lo.y, p1.lo.x, p1.lo.y, p2.lo.x, p2.lo.y, p3.lo.x, p3.lo.y};
  return o;
}

// Operand order. A product's result leaves lane l with rows 4 (l / 16) + r of each 16-row
// tile, in column l % 16. As the next product's right operand those registers are used as
// they are: position (l / 16, j) of a 32-deep step then stands for row 16 (j / 4) +
// 4 (l / 16) + j % 4, and left operands are stored in that order: index x of 32 goes to
// place 8 ((x % 16) / 4) + 4 (x / 16) + x % 4.
__device__ __forceinline__ int place(int x) { return 8 * ((x & 15) >> 2) + 4 * (x >> 4) + (x & 3); }

// The sequence and piece that program p owns: the largest s with v(s) <= p, and p - v(s),
// where v(s) numbers the sequence's first program (see Pieces). A 64-way search, one ballot
// per level. Returns s = -1 when no sequence starts early enough.
struct Piece {
  int s, index;
};

__device__ __forceinline__ Piece find_piece(const ChunkParams& P, const Pieces& pieces, int p, int lane) {
  const RuleParams& R = P.R;
  int base = 0, v = 0;
  for (int stride = P.search_top; stride > 0; stride >>= 6) {
    const int s = base + lane * stride;
    int at = 0;
    bool ok = s < R.num_seqs;
    if (ok) {
      int a = R.qsl[s];
      a = a < 0 ? 0 : (a > R.num_tokens ? R.num_tokens : a);
      at = pieces.first(s, a);
      ok = at <= p;
    }
    const uint64_t mask = __ballot(ok);
    const int n = __builtin_popcountll(mask);
    if (n == 0) return Piece{-1, 0};
    base += (n - 1) * stride;
    v = __shfl(at, n - 1);
  }
  // Offsets out of order may take the search to a sequence whose first program is later.
  const int index = p - uniform(v);
  return index < 0 ? Piece{-1, 0} : Piece{uniform(base), index};
}

// Sequences of up to P.whole_chunks are not cut.
__device__ __forceinline__ int chunks_per_segment(const ChunkParams& P, int chunks) {
  return chunks <= P.whole_chunks ? chunks : P.segment_chunks;
}

// How the prepare kernel's kWaves waves hold a chunk's rows: two channels per lane, in
// groups of 4 neighbouring rows. Of 4 waves wave w has rows 4 w .. and 16 + 4 w .. (one place
// of 8 in the order above): with 128 channels each lane has both groups, with 64 the lanes'
// halves have one each. Of 8 waves (128 channels) wave w has rows 4 w .. . Running sums go
// over these groups.
template <int D, int kWaves>
struct Rows {
  static constexpr int kLanes = D / 2;  // lanes per row
  static constexpr int kParts = kLanes / (8 * kWaves);  // groups of 4 rows per lane
  static constexpr int kRows = 4 * kParts;

  // Row i of a lane: the same for all lanes of a wave, plus the lane's part.
  static __device__ __forceinline__ int wave_row(int wave, int i) { return 4 * wave + i % 4 + 16 * (i / 4); }
  static __device__ __forceinline__ int lane_row(int lane) { return D == 128 ? 0 : lane / 32 * 16; }
  // Whether the lane's group j is in the chunk's second half.
  static __device__ __forceinline__ bool second(int wave, int lane, int j) {
    return kParts == 2 ? j == 1 : (D == 128 ? wave >= 4 : lane >= 32);
  }
};

// Hides that x is the same in every iteration of a loop. Without it the compiler computes
// each row's offset once, before the loop, and keeps all of them in registers, which
// spilled.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Rows of a chunk behind a buffer descriptor that ends with the last valid row: a load past
// it brings zeros and a store past it does nothing, so rows need no branches, and lanes
// need one 32-bit offset (32 rows stay below 2^30 bytes). Rows that share memory (a token
// stride below a row) may still be read past the last: mask_rows.
struct Window {
  __amdgpu_buffer_rsrc_t r;
  uint32_t stride;

  __device__ __forceinline__ Window(const char* base, int valid, uint32_t stride, uint32_t row_bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0,
                                            (int)((valid - 1) * stride + row_bytes), 0x00020000)),
        stride(stride) {}
};

template <int kF>
struct Cell;  // loads of one element or a pair, stores of one

template <>
struct Cell<kRuleF32> {
  static __device__ __forceinline__ f32x2 pair(const Window& w, uint32_t lane, uint32_t row) {
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(w.r, lane, row * w.stride, 0));
  }
  static __device__ __forceinline__ f32x2 one(const Window& w, uint32_t lane, uint32_t row) {
    return f32x2{__builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(w.r, lane, row * w.stride, 0)), 0.0f};
  }
  static __device__ __forceinline__ void store_one(const Window& w, uint32_t lane, uint32_t row, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), w.r, lane, row * w.stride, 0);
  }
};

template <int kF>
struct Cell {
  static __device__ __forceinline__ uint32_t pair(const Window& w, uint32_t lane, uint32_t row) {
    return __builtin_amdgcn_raw_buffer_load_b32(w.r, lane, row * w.stride, 0);
  }
  static __device__ __forceinline__ uint32_t one(const Window& w, uint32_t lane, uint32_t row) {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(w.r, lane, row * w.stride, 0);
  }
  static __device__ __forceinline__ void store_one(const Window& w, uint32_t lane, uint32_t row, float v) {
    uint32_t bits;
    if constexpr (kF == kRuleBF16)
      bits = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, v}, bf16x2));
    else
      bits = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, v}, f16x2));
    __builtin_amdgcn_raw_buffer_store_b16((short)bits, w.r, lane, row * w.stride, 0);
  }
};

// A lane's pairs of its rows, as loaded; `lane` is the lane's offset (its channels, and its
// part of the rows).
template <int kF, class RW>
struct RawRows {
  static constexpr int N = RW::kRows;
  typename Pair<kF>::raw r[N];

  __device__ __forceinline__ void load(const Window& w, uint32_t lane, int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = Cell<kF>::pair(w, lane, RW::wave_row(wave, i));
  }

  // One element per row, for both of the lane's channels (gates per head).
  __device__ __forceinline__ void load_same(const Window& w, uint32_t lane, int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = Cell<kF>::one(w, lane, RW::wave_row(wave, i));
  }

  __device__ __forceinline__ void values(f32x2 (&x)[N], bool same) const {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Pair<kF>::value(r[i]);
    if (same) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i].y = x[i].x;
    }
  }
};

// Zeros in the rows past the last.
template <class RW>
__device__ __forceinline__ void mask_rows(f32x2 (&x)[RW::kRows], int wave, int lane, int valid) {
  if (valid == kChunk) return;
#pragma unroll
  for (int i = 0; i < RW::kRows; ++i)
    if (RW::wave_row(wave, i) + RW::lane_row(lane) >= valid) x[i] = f32x2{0.0f, 0.0f};
}

// Sums of N values over 2 kMask lanes, each lane receiving the sum of value (lane index /
// (2 kMask / N)): exchanges halves while values are left, so N + log2(2 kMask / N) - 1
// exchanges instead of N log2(2 kMask). All are moves inside the vector unit. The values
// travel as a vector: the compiler turns a choice between two elements of an array into a
// choice of the index, which costs more than all the rest.
template <int N>
struct Doubles {
  typedef double type __attribute__((ext_vector_type(N)));
};

typedef uint32_t u32two __attribute__((ext_vector_type(2)));

// x of the lane whose number differs in bit kMask; for 4 the lower bits differ too (which
// lane of its half a value comes from does not matter to a sum over all of them).
template <int kMask>
__device__ __forceinline__ double from_other(double x) {
  constexpr int kMove = kMask == 8 ? 0x128 : kMask == 4 ? 0x141 : kMask == 2 ? 0x4E : 0xB1;
  static_assert(kMask <= 8, "one move inside rows of 16 lanes");
  u32two w = __builtin_bit_cast(u32two, x);
  w.x = (uint32_t)__builtin_amdgcn_mov_dpp((int)w.x, kMove, 0xF, 0xF, true);
  w.y = (uint32_t)__builtin_amdgcn_mov_dpp((int)w.y, kMove, 0xF, 0xF, true);
  return __builtin_bit_cast(double, w);
}

// a + a of the other half of the lanes in the half without bit kMask, the same of b in the
// half with it.
template <int kMask>
__device__ __forceinline__ double halves_sum(double a, double b, int lane) {
  if constexpr (kMask >= 16) {
    const u32two x = __builtin_bit_cast(u32two, a), y = __builtin_bit_cast(u32two, b);
    u32two lo, hi;  // of both words
    if constexpr (kMask == 32) {
      lo = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
      hi = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
    } else {
      lo = __builtin_amdgcn_permlane16_swap(x.x, y.x, false, false);
      hi = __builtin_amdgcn_permlane16_swap(x.y, y.y, false, false);
    }
    return __builtin_bit_cast(double, u32two{lo.x, hi.x}) + __builtin_bit_cast(double, u32two{lo.y, hi.y});
  } else {
    const bool upper = (lane & kMask) != 0;
    return (upper ? b : a) + from_other<kMask>(upper ? a : b);
  }
}

template <int N, int kMask>
__device__ __forceinline__ double scatter_sum(typename Doubles<N>::type x, int lane) {
  if constexpr (N == 2) {
    double s = halves_sum<kMask>(x[0], x[1], lane);
    if constexpr (kMask > 4) s += from_other<4>(s);
    if constexpr (kMask > 2) s += from_other<2>(s);
    return s + from_other<1>(s);
  } else {
    typename Doubles<N / 2>::type y;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) y[i] = halves_sum<kMask>(x[i], x[N / 2 + i], lane);
    return scatter_sum<N / 2, kMask / 2>(y, lane);
  }
}

// ---------------------------------------------------------------------------- prepare

// With 128 channels 4 or 8 waves: of 8 only two workgroups fit a CU (53 KB of LDS, 122
// registers), but each is faster; of 4 three do (162 registers). Of 4 one alone takes about 25000
// cycles: finding its chunk 1600, loads and gates 3900, lengths and sums 1500, operands of the
// products 2400, products 4500, L and A 1300, operands for the scans 3400, T 4600, the rest
// its stores. 6144 of them (16384 tokens, 12 heads of 128) take 147 us for 550 MB, 3.7 TB/s,
// and no single part bounds that: without its stores it takes 15 us less, without the products
// 31, without T 17, without the scans' operands 24, without the checks for values that are not
// finite 2. The way through all of them at three workgroups per CU does; a fourth would need 40 KB
// of LDS and 128 registers.
template <int kF, int kG, int D, int kWaves>
__global__ __launch_bounds__(64 * kWaves, kWaves == 8 ? 4 : 3) void delta_rule_prepare_kernel(const ChunkParams P) {
  typedef Rows<D, kWaves> RW;
  constexpr int kThreads = 64 * kWaves;
  constexpr int kRows = RW::kRows, kLanes = RW::kLanes, kParts = RW::kParts;
  constexpr int kEB = elem_bytes<kF>(), kGB = elem_bytes<kG>();
  constexpr int kLd = D + 4;  // floats per operand row: 16 rows reach all banks
  constexpr int kMat = kChunk * kLd;
  constexpr int kSq = 34;  // doubles per row of a 32 x 32 matrix
  // After the products: L and its inverse, A's parts, and 128 D bytes to turn rows
  // into operands.
  constexpr int kSquares = 2 * kChunk * kSq * (int)sizeof(double), kStage = kSquares + 4096;
  constexpr int kBytes = 3 * kMat * 4 > kStage + 128 * D ? 3 * kMat * 4 : kStage + 128 * D;
  // Operand rows q, k (times the decay from the block's middle) and columns k.
  __shared__ __attribute__((aligned(16))) char shared[kBytes];
  // The groups' decays, read before the operands take their place.
  float (*const tot)[D] = (float (*)[D])shared;
  // Decays of a chunk's second 8 tokens and of its third.
  __shared__ __attribute__((aligned(16))) float across[2][D];
  // Per row: the key's factor times 16, the query's times 16, the key's power of two; and
  // as they go to the slot |k| / 16 and the outputs' factor / 16.
  __shared__ float kf16[kChunk], qf16[kChunk], ktwo[kChunk];
  __shared__ __attribute__((aligned(16))) float rows[2][kChunk];
  __shared__ int texp;  // T's scale is 2 to this
  __shared__ float beta[kChunk];
  // Keys enter the products times a power of two (exact); the rest of their factor, and n,
  // follow in FP64 (a key rounded to unit length would be off by 3e-8, see below).
  __shared__ float krest[kChunk];
  __shared__ double kfac[kChunk];
  __shared__ int steep;
  __shared__ int unfinite[kWaves];  // each wave's first row with a value that is not finite
  float* const mq = (float*)shared;
  float* const mk = mq + kMat;
  float* const mc = mq + 2 * kMat;

  const RuleParams& R = P.R;
  const int program = blockIdx.x / R.heads, h = blockIdx.x % R.heads;
  const int wave = uniform(threadIdx.x / kRuleWave), lane = threadIdx.x % kRuleWave;
  const Piece piece = find_piece(P, P.chunk_pieces, program, lane);
  if (piece.s < 0) return;
  const Sequence seq(R, piece.s);
  if (seq.len < P.min_len || piece.index * kChunk >= seq.len) return;
  const int64_t first = seq.start + piece.index * kChunk;
  const int valid = seq.len - piece.index * kChunk < kChunk ? seq.len - piece.index * kChunk : kChunk;

  const int c = 2 * (lane % kLanes), lrow = RW::lane_row(lane);
  const int quad = wave % 4;  // the lane's rows are 4 quad .. of their blocks of 16
  const int64_t qk = h / R.share;
  const Window wq(R.q + (first * R.q_ts + qk * R.q_hs) * kEB, valid, (uint32_t)R.q_ts * kEB, D * kEB);
  const Window wk(R.k + (first * R.k_ts + qk * R.k_hs) * kEB, valid, (uint32_t)R.k_ts * kEB, D * kEB);
  const Window wg(R.g + (first * R.g_ts + h * R.g_hs) * kGB, valid, (uint32_t)R.g_ts * kGB,
                  (R.g_cs != 0 ? D : 1) * kGB);
  const auto load_gates = [&](RawRows<kG, RW>& rg) {
    if (R.g_cs != 0)
      rg.load(wg, lrow * wg.stride + c * kGB, wave);
    else
      rg.load_same(wg, lrow * wg.stride, wave);
  };

  const Gate gate(R, h);
  f32x2 bias = {0.0f, 0.0f};
  if (R.dt_bias != nullptr) bias = *(const f32x2a4*)(R.dt_bias + h * D + c);
  // The lane's log2 decays, zeros from row `end` on.
  const auto read_gates = [&](f32x2 (&g)[kRows], int end) {
    RawRows<kG, RW> rg;
    load_gates(rg);
    rg.values(g, R.g_cs == 0);
    gate.eval(g, bias);
    mask_rows<RW>(g, wave, lane, end);
  };

  f32x2 q[kRows], k[kRows], p[kRows];  // p: log2 decays, then their running sums
  f32x2 rest[kRows];  // log2 decay after each row, inside its group of 4
  {
    RawRows<kF, RW> rq, rk;
    RawRows<kG, RW> rg;
    load_gates(rg);
    rk.load(wk, lrow * wk.stride + c * kEB, wave);
    rq.load(wq, lrow * wq.stride + c * kEB, wave);
    rg.values(p, R.g_cs == 0);
    rk.values(k, false);
    mask_rows<RW>(k, wave, lane, valid);
    rq.values(q, false);
    mask_rows<RW>(q, wave, lane, valid);
    gate.eval(p, bias);
    mask_rows<RW>(p, wave, lane, valid);
  }
  int odd = kChunk;  // the first row here with a key or a step that is not finite
  if (threadIdx.x < kChunk) {
    const float b = (int)threadIdx.x < valid ? beta_value(R, kF, first + threadIdx.x, h) : 0.0f;
    beta[threadIdx.x] = b;
    if (!is_finite(b)) odd = threadIdx.x;
  }
  if (threadIdx.x == 0) steep = 0;

  // Lengths of the rows' queries and keys.
  {
    typename Doubles<2 * kRows>::type ss;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const double qx = q[i].x, qy = q[i].y, kx = k[i].x, ky = k[i].y;
      ss[i] = __builtin_fma(qx, qx, qy * qy);
      ss[kRows + i] = __builtin_fma(kx, kx, ky * ky);
    }
    const double s = scatter_sum<2 * kRows, kLanes / 2>(ss, lane);
    constexpr int kShare = kLanes / (2 * kRows);  // lanes holding the same sum
    const int l = lane % kLanes, which = l / kShare, r = RW::wave_row(wave, which % kRows) + lrow;
    if (l % kShare == 0) {
      // Of a row that is 0.7 long or longer after its normalisation the products take it as it is.
      // Other rows, and those taken without normalisation, enter them at unit length (or 2^118
      // times themselves, the shortest) and n is the rest: pairs of FP16 values would lose a row
      // that vanishes beside l2_eps.
      const bool norm = R.l2_eps >= 0.0f;
      const double eps = R.l2_eps, least = 0x1p-236;
      const bool whole = norm && s >= eps && s >= least;
      const double own = s < least ? least : s, back = inverse_root_f64(whole ? s + eps : own);
      const Factor f = two_floats(back);
      const float n = whole ? 1.0f : (float)(norm ? own * back * inverse_root_f64(s + eps) : own * back);
      if (which < kRows) {
        qf16[r] = kVec * f.hi;
        rows[1][r] = n * R.scale * (1.0f / kVec);
      } else {
        kf16[r] = kVec * f.hi;
        rows[0][r] = n * (1.0f / kVec);
        const int e = f.hi > 0.0f ? __builtin_amdgcn_frexp_expf(f.hi) : 0;
        ktwo[r] = __builtin_amdgcn_ldexpf(1.0f, e);
        krest[r] = __builtin_amdgcn_ldexpf(f.hi, -e);
        kfac[r] = (double)n * __builtin_amdgcn_ldexp((double)f.hi + (double)f.lo, -e);
        if (!(s < __builtin_huge_val())) odd = odd < r ? odd : r;
      }
    }
  }
  // Running sums inside the groups.
  const auto running_sums = [&]() {
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      rest[4 * j + 3] = f32x2{0.0f, 0.0f};
#pragma unroll
      for (int i = 3; i > 0; --i) rest[4 * j + i - 1] = rest[4 * j + i] + p[4 * j + i];
#pragma unroll
      for (int i = 1; i < 4; ++i) p[4 * j + i] += p[4 * j + i - 1];
      *(f32x2*)&tot[4 * RW::second(wave, lane, j) + quad][c] = p[4 * j + 3];
    }
  };
  running_sums();
  // A key, step or decay that is not finite makes all values from its token on NaN, and none
  // before: the matrix products would carry it there (0 times NaN). The chunk ends before that
  // token as far as they are concerned, and n says NaN from there on, which the scans see.
  {
    bool any = odd < kChunk;
#pragma unroll
    for (int j = 0; j < kParts; ++j) any |= !(is_finite(p[4 * j + 3].x) && is_finite(p[4 * j + 3].y));
    if (__ballot(any) != 0) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = RW::wave_row(wave, i) + lrow;
        if (!(is_finite(p[i].x) && is_finite(p[i].y))) odd = odd < r ? odd : r;
      }
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) {
        const int other = __shfl_xor(odd, m);
        odd = odd < other ? odd : other;
      }
    }
    if (lane == 0) unfinite[wave] = odd;
  }
  __syncthreads();
  int live = valid;  // rows before it
#pragma unroll
  for (int w = 0; w < kWaves; ++w) live = live < unfinite[w] ? live : unfinite[w];
  live = uniform(live);
  if (live < valid) {
    read_gates(p, live);
    running_sums();
    mask_rows<RW>(k, wave, lane, live);
    if (threadIdx.x < kChunk && (int)threadIdx.x >= live)
      beta[threadIdx.x] = kf16[threadIdx.x] = ktwo[threadIdx.x] = krest[threadIdx.x] = rows[0][threadIdx.x] =
          kfac[threadIdx.x] = 0.0f;
    __syncthreads();
  }

  // Each block of 16 rows takes its decays from its middle (after 8 rows): rows carry 2^d and
  // columns 2^-d, where d is the log2 decay from the middle to the row. That stays in range
  // while both halves of the block are within 2^101 (8 tokens of log decay -8.75 each; the
  // bounded gate reaches -5); steeper chunks take the direct sums below. d is summed from the
  // middle outwards: rows nearer to the middle than a strong decay do not carry it, and the
  // product of a row and a column of these is exact to a few 2^-24. Rows beyond it do, and
  // each addition to a sum of up to 101 is off by up to 2^-18, which the product then is too.
  // Between the blocks lie the decays of block 0's second half and of block 1's first. Their
  // product may leave FP32's range where neither does, so columns of block 0 carry one and rows
  // of block 1 the other: each scaled operand is at most its vector.
  f32x2 all[2], mid[2], late[2];  // of both blocks; late: of their second halves
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const f32x2 t0 = *(const f32x2*)&tot[4 * b][c], t1 = *(const f32x2*)&tot[4 * b + 1][c];
    const f32x2 t2 = *(const f32x2*)&tot[4 * b + 2][c], t3 = *(const f32x2*)&tot[4 * b + 3][c];
    mid[b] = t0 + t1;
    late[b] = t2 + t3;
    all[b] = mid[b] + late[b];
    if (mid[b].x < -101.0f || mid[b].y < -101.0f || late[b].x < -101.0f || late[b].y < -101.0f) steep = 1;
  }
  // Log2 decays of the block before and after the group, and between it and the middle.
  f32x2 before[kParts], after[kParts], inner[kParts];
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    before[j] = after[j] = inner[j] = f32x2{0.0f, 0.0f};
    const int b = RW::second(wave, lane, j);
    if (quad == 0 || quad == 3) inner[j] = *(const f32x2*)&tot[4 * b + (quad == 0 ? 1 : 2)][c];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 t = *(const f32x2*)&tot[4 * b + i][c];
      if (i < quad) before[j] += t;
      if (i > quad) after[j] += t;
    }
  }
  if (wave == 0 && lane < kLanes) {
    *(f32x2*)&across[0][c] = f32x2{exp2_hw(late[0].x), exp2_hw(late[0].y)};
    *(f32x2*)&across[1][c] = f32x2{exp2_hw(mid[1].x), exp2_hw(mid[1].y)};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = RW::wave_row(wave, i) + lrow, j = i / 4;
    const f32x2 d = quad < 2 ? -(rest[i] + inner[j]) : p[i] + inner[j];
    const f32x2 e = {exp2_hw(d.x), exp2_hw(d.y)}, m = {exp2_hw(-d.x), exp2_hw(-d.y)};
    const f32x2 kk = k[i] * ktwo[r];
    *(f32x2*)&mq[r * kLd + c] = q[i] * qf16[r] * e;
    *(f32x2*)&mk[r * kLd + c] = kk * e;
    *(f32x2*)&mc[r * kLd + c] = kk * m;
  }
  __syncthreads();

  const int n16 = lane % 16, n4 = lane / 16;
  f64x4 akk = {0.0, 0.0, 0.0, 0.0};  // kinds 0 to 2: one 16 x 16 block of key products each
  f32x4 aqk[3] = {};  // kind 3: all three of queries and keys
  // Of 8 waves two share a kind, half of the channels each.
  const int kind = kWaves == 8 ? (wave < 6 ? wave % 3 : 3) : wave;
  const int part = kWaves == 8 ? (wave < 6 ? wave / 3 : wave - 6) : 0;
  constexpr int kShared = kWaves == 8 ? D / 2 : D;
  double dkk[3];
  float dqk[3];
  const bool direct = steep != 0;
  if (!direct) {
    // Blocks (row, column): 0 (0, 0), 1 (1, 1), 2 (1, 0). The key products are summed in
    // FP64: equal keys with steps near 2 (reflections) and no decay make an error common to
    // L's entries grow with the tokens, by 32 per chunk. FP32 sums and an FP32 inverse left
    // such a state 1e-4 off after 97 tokens. Both kinds take as long: 125 cycles for an FP64
    // instruction, 46 for one of the three times as many FP32 ones of kind 3.
    const int from = kShared * part + 4 * n4;
    if (kind < 3) {
      const float* const rk = mk + ((kind == 0 ? 0 : 16) + n16) * kLd + from;
      const float* const rc = mc + ((kind == 1 ? 16 : 0) + n16) * kLd + from;
#pragma unroll
      for (int b = 0; b < kShared; b += 16) {
        f32x4 x = *(const f32x4*)(rk + b), z = *(const f32x4*)(rc + b);
        if (kind == 2) {
          x *= *(const f32x4*)&across[1][b + from];
          z *= *(const f32x4*)&across[0][b + from];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) akk = mfma64((double)x[e], (double)z[e], akk);
      }
    } else {
      const float* const rq = mq + n16 * kLd + from;
      const float* const rc = mc + n16 * kLd + from;
#pragma unroll
      for (int b = 0; b < kShared; b += 16) {
        const f32x4 x0 = *(const f32x4*)(rq + b), x1 = *(const f32x4*)(rq + 16 * kLd + b);
        const f32x4 z0 = *(const f32x4*)(rc + b), z1 = *(const f32x4*)(rc + 16 * kLd + b);
        const f32x4 x2 = x1 * *(const f32x4*)&across[1][b + from];
        const f32x4 z2 = z0 * *(const f32x4*)&across[0][b + from];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          aqk[0] = mfma32(x0[e], z0[e], aqk[0]);
          aqk[1] = mfma32(x1[e], z1[e], aqk[1]);
          aqk[2] = mfma32(x2[e], z2[e], aqk[2]);
        }
      }
    }
  } else {
    // Direct sums of k_t k_i 2^(G_t - G_i), with the running sums G in FP64 (a chunk may
    // hold many resets, and FP32 sums of -150 each would lose the small decays between). The
    // key products are summed in FP64 as above: the chunk may hold reflections in its other
    // channels.
    __syncthreads();
    // The decays, from the sums: exact enough again, then summed in FP64 per channel.
    {
      f32x2 g[kRows];
      read_gates(g, live);
#pragma unroll
      for (int i = 0; i < kRows; ++i) *(f32x2*)&mk[(RW::wave_row(wave, i) + lrow) * kLd + c] = g[i];
    }
    __syncthreads();
    double* const sums = (double*)mc;  // rows of D doubles over mc and mq's place
    static_assert(sizeof(double) * kChunk * D <= sizeof(float) * 2 * kMat, "FP64 sums fit");
    double* const lower = (double*)mq;
    // Rows 0-15 in mc, rows 16-31 in mq (each 16 D doubles <= kMat floats).
    if (threadIdx.x < D) {
      double s = 0.0;
      for (int r = 0; r < kChunk; ++r) {
        s += (double)mk[r * kLd + threadIdx.x];
        (r < 16 ? sums : lower)[(r & 15) * D + threadIdx.x] = s;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = RW::wave_row(wave, i) + lrow;
      *(f32x2*)&mk[r * kLd + c] = k[i] * ktwo[r];
    }
    __syncthreads();
    for (int u = 0; u < 3; ++u) {
      const int pair = threadIdx.x + kThreads * u;  // (t, i) with i <= t, 528 in all
      dkk[u] = 0.0;
      dqk[u] = 0.0f;
      if (pair >= 528) continue;
      int t = 0;
      while ((t + 1) * (t + 2) / 2 <= pair) ++t;
      const int i = pair - t * (t + 1) / 2;
      const double* const gt = (t < 16 ? sums : lower) + (t & 15) * D;
      const double* const gi = (i < 16 ? sums : lower) + (i & 15) * D;
      const char* const qrow =
          R.q + ((first + (t < valid ? t : valid - 1)) * R.q_ts + qk * R.q_hs) * kEB;
      const float fq = t < valid ? qf16[t] : 0.0f;
      double sk = 0.0;
      float sq = 0.0f;
      for (int ch = 0; ch < D; ++ch) {
        const float w = mk[i * kLd + ch] * exp2_hw((float)(gt[ch] - gi[ch]));
        sk = __builtin_fma((double)mk[t * kLd + ch], (double)w, sk);
        sq = __builtin_fmaf(load_elem<kF>(qrow + ch * kEB) * fq, w, sq);
      }
      dkk[u] = sk;
      dqk[u] = t < valid ? sq : 0.0f;
    }
  }
  __syncthreads();

  // The operands are done with; their place takes L, the inverse and the staged outputs.
  double* const ml = (double*)shared;  // L [row][column]
  double* const mt = ml + kChunk * kSq;  // (I + L)^-1
  _Float16* const sa = (_Float16*)(shared + kSquares);  // A in two parts, as it goes to the slot
  constexpr Slot kSlot{D};
  char* const slot = P.slots + ((int64_t)program * R.heads + h) * kSlot.bytes();
  const auto put_a = [&](int t, int i, float a) {
    // A times 256 in operand order: row tile, lane, place. (a carries the query's 16.)
    const int at = (t / 16 * 64 + (place(i) / 8) * 16 + t % 16) * 8 + place(i) % 8;
    const float x = 16.0f * krest[i] * a;
    const _Float16 hi = (_Float16)x;
    sa[at] = hi;
    sa[1024 + at] = (_Float16)(x - (float)hi);
  };
  const auto put_l = [&](int t, int i, double a) {
    ml[t * kSq + i] =
        i < t ? (double)beta[t] * (kfac[t] * kfac[i]) * a : 0.0;
  };
  if (!direct) {
    // FP64 results: register r of lane l is row 4 r + l / 16.
    const int rows = kind == 0 ? 0 : 16, cols = kind == 1 ? 16 : 0;
    if (kWaves == 8) {
      // The second parts come through the inverse's place and the staging area.
      float* const aside = (float*)(shared + kStage) + lane;
      if (part == 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (kind < 3)
            mt[(rows + 4 * r + n4) * kSq + cols + n16] = akk[r];
          else
#pragma unroll
            for (int b = 0; b < 3; ++b) aside[64 * (4 * b + r)] = aqk[b][r];
        }
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (kind < 3)
            akk[r] += mt[(rows + 4 * r + n4) * kSq + cols + n16];
          else
#pragma unroll
            for (int b = 0; b < 3; ++b) aqk[b][r] += aside[64 * (4 * b + r)];
        }
      }
    }
    if (part == 0) {
      if (kind < 3) {
#pragma unroll
        for (int r = 0; r < 4; ++r) put_l(rows + 4 * r + n4, cols + n16, akk[r]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 4 * n4 + r;
          put_a(t, n16, n16 <= t ? aqk[0][r] : 0.0f);
          put_a(16 + t, 16 + n16, n16 <= t ? aqk[1][r] : 0.0f);
          put_a(16 + t, n16, aqk[2][r]);
          put_a(t, 16 + n16, 0.0f);
        }
      }
    }
  } else {
    for (int u = 0; u < 3; ++u) {
      const int pair = threadIdx.x + kThreads * u;
      if (pair >= 528) continue;
      int t = 0;
      while ((t + 1) * (t + 2) / 2 <= pair) ++t;
      const int i = pair - t * (t + 1) / 2;
      put_l(t, i, dkk[u]);
      put_a(t, i, dqk[u]);
      if (i < t) put_a(i, t, 0.0f);
    }
  }
  __syncthreads();

  // The scans' operands.
  {
    // The wave's pieces of a row matrix: (32 channels, 16 rows, hi or lo), of both row tiles or
    // of 8 waves of one.
    constexpr int kTiles = kWaves == 8 ? 1 : 2, kFrags = D / 32 * kTiles * 2;
    _Float16* const own = (_Float16*)(shared + kStage + kFrags * 256 * wave);
    const int x = c % 32, kk = c / 32, place16 = place(x);
    f16x2 th[kRows], tl[kRows];
    HalfPair qs[kRows];
    // The wave's 4 rows of a row tile and 4 channels of 8 make 4 x 4 blocks of 16 bytes per
    // operand piece; block (channels n, row r) sits at 4 n + (r ^ n), xor the piece's number
    // of 32 channels, so that a row's 64 lanes reach all banks.
    const auto own_at = [&](int i, int part) {
      const int tt = kTiles == 2 ? RW::second(wave, lane, i / 4) : 0, n = place16 / 8, r = i % 4;
      return ((kk * kTiles + tt) * 2 + part) * 128 + (((4 * n + (r ^ n)) ^ kk) * 8) + place16 % 8;
    };
    const auto copy_out = [&](char* to) {
#pragma unroll
      for (int f0 = 0; f0 < kFrags; f0 += 4) {
        const int f = f0 + lane / 16, b = lane % 16, fk = f / (2 * kTiles);
        const int tt = kTiles == 2 ? f / 2 % 2 : wave / 4;
        const u32q v = *(const u32q*)(own + f * 128 + ((b ^ fk) * 8));
        // In the slot block (channels n, row r of 16) of a piece is 16 n + (r ^ (n + 4 kk)).
        *(u32q*)(to + ((2 * fk + tt) * 2 + f % 2) * 1024 + (16 * (b / 4) + 4 * (quad ^ fk) + b % 4) * 16) = v;
      }
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = RW::wave_row(wave, i) + lrow, j = i / 4;
      const bool second = RW::second(wave, lane, j);
      const f32x2 up = p[i] + before[j] + (second ? all[0] : f32x2{0.0f, 0.0f});
      const f32x2 down = rest[i] + after[j] + (second ? f32x2{0.0f, 0.0f} : all[1]);
      const f32x2 e = {exp2_hw(up.x), exp2_hw(up.y)};
      const f32x2 unit = k[i] * kf16[r];
      const HalfPair g = split2(unit * e, R.one);
      *(f16x2*)&own[own_at(i, 0)] = g.hi;
      *(f16x2*)&own[own_at(i, 1)] = g.lo;
      qs[i] = split2(q[i] * qf16[r] * e, R.one);
      const HalfPair t = split2(unit * f32x2{exp2_hw(down.x), exp2_hw(down.y)}, R.one);
      th[i] = t.hi;
      tl[i] = t.lo;
    }
    __builtin_amdgcn_wave_barrier();
    copy_out(slot + kSlot.kg());
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      *(f16x2*)&own[own_at(i, 0)] = qs[i].hi;
      *(f16x2*)&own[own_at(i, 1)] = qs[i].lo;
    }
    __builtin_amdgcn_wave_barrier();
    copy_out(slot + kSlot.qg());
    // Columns: a channel's rows 4 quad .. of both blocks of 16 are one block of 16 bytes.
    _Float16* const kt = (_Float16*)(slot + kSlot.kt());
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int ch = c + y, row = (ch / 16) * 1024 + (16 * quad + ch % 16) * 8;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        const int at = row + 4 * RW::second(wave, lane, j);
        f16x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = th[4 * j + i][y];
          lo[i] = tl[4 * j + i][y];
        }
        *(f16x4*)&kt[at] = hi;
        *(f16x4*)&kt[at + 512] = lo;
      }
    }
    if (wave == 0) {
      const f32x2 d = all[0] + all[1], e = {exp2_hw(d.x), exp2_hw(d.y)};
      if (lane < kLanes) *(f32x2*)(slot + kSlot.factors() + 4 * c) = e;
      const bool keeps = __ballot(e.x >= kFaded || e.y >= kFaded) != 0;
      if (lane == 0) ((float*)(slot + kSlot.factors()))[kFactorFaded] = keeps ? 1.0f : 0.0f;
    }
  }

  if (wave == 0) {
    // (I + L)^-1 in FP64. Four 8 x 8 diagonal blocks by forward substitution, a column per
    // lane; then twice from blocks A, B on the diagonal and C below to the inverse of
    // [A 0; C B], whose lower left is -B^-1 (C A^-1). A result's registers (row 4 r +
    // lane / 16) are the next product's right operand as they are.
    if (lane < 32) {
      const int b = lane & 24, col = lane & 7;
      double x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        double s = t == col ? 1.0 : 0.0;
#pragma unroll
        for (int i = 0; i < t; ++i) s = __builtin_fma(-ml[(b + t) * kSq + b + i], x[i], s);
        x[t] = s;
        mt[(b + t) * kSq + b + col] = s;
      }
    }
    __builtin_amdgcn_wave_barrier();
    f64x4 t00, t11, t10 = {0.0, 0.0, 0.0, 0.0};
    {
      const bool diagonal = (n16 & 8) == 0;  // this lane's column is in the first 8
      f64x4 w[2], y[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        w[b] = y[b] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = 16 * b + n16, at = 16 * b + 4 * k + n4;
          const double c = n16 >= 8 ? ml[row * kSq + at] : 0.0;
          w[b] = mfma64(c, diagonal ? mt[at * kSq + row] : 0.0, w[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 2; k < 4; ++k) {
          const double x = n16 >= 8 ? mt[(16 * b + n16) * kSq + 16 * b + 4 * k + n4] : 0.0;
          y[b] = mfma64(x, w[b][k], y[b]);
        }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // Registers 0 and 1 are rows 0 to 7.
        const bool own = (r < 2) == diagonal;
        const int at = (4 * r + n4) * kSq + n16;
        t00[r] = own ? mt[at] : -y[0][r];
        t11[r] = own ? mt[at + 16 * kSq + 16] : -y[1][r];
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 4; ++r) mt[(16 + 4 * r + n4) * kSq + 16 + n16] = t11[r];
    __builtin_amdgcn_wave_barrier();
    {
      f64x4 w = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int k = 0; k < 4; ++k) w = mfma64(ml[(16 + n16) * kSq + 4 * k + n4], t00[k], w);
#pragma unroll
      for (int k = 0; k < 4; ++k) t10 = mfma64(mt[(16 + n16) * kSq + 16 + 4 * k + n4], w[k], t10);
    }
    __builtin_amdgcn_wave_barrier();
    // diag(n) T diag(b), and its largest entry.
    float top = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * r + n4;
      const double n0 = (double)(kVec * rows[0][t]), n1 = (double)(kVec * rows[0][16 + t]);
      const double b0 = (double)beta[n16], b1 = (double)beta[16 + n16];
      const double x0 = n0 * t00[r] * b0, x1 = n1 * t11[r] * b1, x2 = -n1 * t10[r] * b0;
      mt[t * kSq + n16] = x0;
      mt[(16 + t) * kSq + 16 + n16] = x1;
      mt[(16 + t) * kSq + n16] = x2;
      top = __builtin_fmaxf(top, __builtin_fmaxf(__builtin_fabsf((float)x2),
                                                 __builtin_fmaxf(__builtin_fabsf((float)x0), __builtin_fabsf((float)x1))));
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, m));
    int e = 0;
    if (top > 0.0f && top < __builtin_huge_valf()) e = 9 - __builtin_amdgcn_frexp_expf(top);
    e = e > 100 ? 100 : e;
    if (lane == 0) texp = e;
  }
  __syncthreads();
  float* const df = (float*)(slot + kSlot.factors());
  if (threadIdx.x < 256) {
    // T scaled to a largest entry of 256 to 512, in three FP16 parts: with two (22 bits) the
    // reflections above still lost 1e-5. Thread u holds places 4 u .. + 3 of the operand
    // order: four neighbouring columns of one row.
    const int u = threadIdx.x, t = (u >> 7) * 16 + ((u >> 1) & 15), i0 = 16 * (u & 1) + 4 * ((u >> 5) & 3);
    const int e = texp;
    f16x4 hi, lo, last;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double x = t < 16 && i0 >= 16 ? 0.0 : __builtin_amdgcn_ldexp(mt[t * kSq + i0 + j], e);
      hi[j] = (_Float16)(float)x;
      const float rest = (float)(x - (double)(float)hi[j]);
      lo[j] = (_Float16)rest;
      last[j] = (_Float16)(rest - (float)lo[j]);
    }
    f16x4* const to = (f16x4*)(slot + kSlot.t()) + u;
    to[0] = hi;
    to[256] = lo;
    to[512] = last;
    // U is kept times 1 / 16, so that (16 k^)^T (U / 16) adds to S as it is.
    if (u == 0) df[kFactorT] = __builtin_amdgcn_ldexpf(1.0f / kVec, -e);
    ((u32q*)(slot + kSlot.a()))[u] = ((const u32q*)sa)[u];
  }
  if (threadIdx.x < 2 * kChunk)
    df[kFactorRows + threadIdx.x] = (int)threadIdx.x >= live && (int)threadIdx.x < valid
                                        ? __builtin_nanf("") : (&rows[0][0])[threadIdx.x];
}

// ------------------------------------------------------------------------------- scan

// The largest magnitude of a column over its 4 lanes.
__device__ __forceinline__ float column_max(float x) {
  x = __builtin_fmaxf(x, __shfl_xor(x, 16));
  return __builtin_fmaxf(x, __shfl_xor(x, 32));
}

// What the scan is run for.
constexpr int kScanOut = 0;  // outputs and final states
constexpr int kScanMove = 1;  // a segment's B and M

// Columns' largest values stay in this range. FP16 ends at 2^16, and its steps at 2^-24: the pairs'
// errors are 2^-28 of the largest value at its lower end.
constexpr float kColLow = 8.0f, kColHigh = 32768.0f;
// And come to 2^6 .. 2^7 when they leave it: X is often 2^4 to 2^8 times S and would be above most
// times if S came to 2^7 .. 2^8 of a range up to 2^13 (16384 tokens 378 us against 373).
constexpr int kColExp = 7;
constexpr int kMostScale = 118;

// 16 columns per wave; lane l holds rows 4 (l / 16) .. + 3 of each 16 of column l % 16.
template <int kM>
struct ScanState {
  f32x4 s[kM];  // times the column's scale
  float scale, inverse;

  __device__ __forceinline__ float largest() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) m = __builtin_fmaxf(m, __builtin_fabsf(s[i][r]));
    return m;
  }

  // Whether some column's values (lanes hold m as their largest) are all below its range.
  static __device__ __forceinline__ bool below(float m) {
    uint64_t big = __ballot(m >= kColLow);
    big |= big >> 32;
    big |= big >> 16;
    return (big & 0xFFFF) != 0xFFFF;
  }

  // Whether all columns' values are below its upper end, and none is NaN.
  static __device__ __forceinline__ bool within(float m) { return __ballot(!(m < kColHigh)) == 0; }

  // The factor that brings a column whose largest value is m back (m from all its lanes).
  __device__ __forceinline__ float factor(float m) const {
    if (!(m > 0.0f) || !(m < __builtin_huge_valf())) return 1.0f;
    if (m >= kColLow && m < kColHigh) return 1.0f;
    // The scale stays at most 2^kMostScale: a column that fades for long would take it to
    // infinity (its values then go to zero as they are).
    const int most = kMostScale + 1 - __builtin_amdgcn_frexp_expf(scale);
    int e = kColExp - __builtin_amdgcn_frexp_expf(m);
    e = e < most ? e : most;
    return __builtin_amdgcn_ldexpf(1.0f, e < 100 ? e : 100);  // (S itself may be far above m)
  }

  __device__ __forceinline__ void apply(float f) {
#pragma unroll
    for (int i = 0; i < kM; ++i) s[i] *= f;
    scale *= f;
    inverse *= rcp_hw(f);  // exact for powers of two
  }
};

// Chunk by chunk with S in registers. Operands come from the slot to LDS by direct loads: the
// row matrices for the next chunk while this chunk's S is updated, the rest while the next
// chunk's products with S run; two barriers per chunk. Waves share the operands and own 16
// columns each; for a segment's transition half of the waves for B and half for M, or (kParts 2)
// one of two workgroups each. (With 32 columns per wave the operands are read from LDS half as
// often, but the 172 matrix instructions per chunk of a lone wave took 24 cycles each instead of
// 14: 20% longer with one sequence of 64 tokens, 5% with many. Two workgroups for the outputs of
// a segment, half of the columns each, took 37 us against 32 for 96 chains of up to 10 chunks.)
//
// 264 output scans of 24 chunks take 99 us: 490 MB, 4.9 TB/s, what a copy reaches; the matrix
// units are busy for 38% of it. The 252 transitions take 113 us for half the bytes:
// 16 waves read 640 KB of operands from LDS per chunk, which is 5000 of its 10000 cycles, and
// the matrix units are busy for 40%.
template <int kF, int D, int kMode, int kParts>
__global__ __launch_bounds__((kMode == kScanOut ? 4 : 8) * D / kParts, 4) void delta_rule_scan_kernel(const ChunkParams P) {
  constexpr bool kOut = kMode == kScanOut;
  constexpr int kColWaves = D / 16, kWaves = (kOut ? 1 : 2) * kColWaves / kParts;
  constexpr int kEB = elem_bytes<kF>();
  constexpr int kM = D / 16, kK = D / 32;
  constexpr Slot kSlot{D};
  constexpr int kMatrix = (int)kSlot.matrix();
  __shared__ __attribute__((aligned(16))) char krows[kMatrix];
  __shared__ __attribute__((aligned(16))) char qrows[kOut ? kMatrix : 16];
  // K^T, factors, T and, for outputs, A, as in the slot.
  __shared__ __attribute__((aligned(16))) char rest[kMatrix + 1024 + 6144 + (kOut ? 4096 : 0)];
  __shared__ float part[8];

  const RuleParams& R = P.R;
  const int program = blockIdx.x / R.heads, h = blockIdx.x % R.heads;
  const int wave = uniform(threadIdx.x / kRuleWave), lane = threadIdx.x % kRuleWave;
  const Piece piece = find_piece(P, kOut ? P.segment_pieces : P.move_pieces, program, lane);
  if (piece.s < 0) return;
  const Sequence seq(R, piece.s);
  if (kOut && seq.len == 0 && P.min_len == 1 && seq.line >= 0 && !seq.init && piece.index == 0) {
    // Without tokens a sequence that starts from zeros leaves them.
    float* const to = R.states + seq.line * R.st_line + h * R.st_head;
    for (int i = threadIdx.x; i < D * D; i += kRuleWave * kWaves) to[i] = 0.0f;
  }
  if (seq.len < P.min_len) return;
  const int chunks = (seq.len + kChunk - 1) / kChunk;
  const int per = chunks_per_segment(P, chunks);
  const int begin = piece.index * per, end = begin + per < chunks ? begin + per : chunks;
  if (begin >= chunks) return;
  if (!kOut && end == chunks) return;

  const int n16 = lane % 16, n4 = lane / 16;
  // This wave's columns are M's; and which.
  const bool identity = !kOut && (kParts == 2 ? blockIdx.y == 1 : wave >= kColWaves);
  const int cw = wave % kColWaves;
  const int col = 16 * cw + n16;
  if (kParts == 2 && identity && begin == 0) return;  // nobody needs the first segment's M
  // The segment's end; for outputs the end of the segment before.
  const int move = kOut ? P.move_pieces.first(piece.s, seq.start) + piece.index - 1 : program;
  const int64_t cell = (int64_t)move * R.heads + h;

  const char* slot = P.slots + ((int64_t)(P.chunk_pieces.first(piece.s, seq.start) + begin) * R.heads + h) * kSlot.bytes();
  const int64_t slot_step = R.heads * kSlot.bytes();
  const auto copy = [&](const char* from, char* to, int pieces) {
#pragma unroll
    for (int i = 0; i < pieces; i += kWaves)
      if (i + wave < pieces) to_lds<kOut>(from + 1024 * (i + wave) + 16 * lane, to + 1024 * (i + wave));
  };
  const auto load_rows = [&](const char* from) {
    copy(from + kSlot.kg(), krows, kMatrix / 1024);
    if (kOut) copy(from + kSlot.qg(), qrows, kMatrix / 1024);
  };
  const auto load_rest = [&](const char* from) {
    copy(from + kSlot.kt(), rest, kMatrix / 1024 + 7 + (kOut ? 4 : 0));
  };
  load_rows(slot);
  load_rest(slot);

  ScanState<kM> S;
  float most;  // the largest magnitude among the lane's values
  {
    const float* from = nullptr;
    if (begin == 0) {
      // Of several segments the last one's outputs may end first, and with them the state:
      // the first then starts from a copy, which the scan of its end leaves in M's place.
      if (seq.init && kOut && chunks > per)
        from = (const float*)(P.moves + (cell + R.heads) * move_bytes(D));
      else if (seq.init)
        from = R.states + seq.line * R.st_line + h * R.st_head;
    } else if (kOut) {
      from = P.ends + cell * (D * D);
    }
    if (from != nullptr && !identity) {
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) S.s[m][r] = from[(16 * m + 4 * n4 + r) * D + col];
      if (!kOut) {
        float* const copy_to = (float*)(P.moves + cell * move_bytes(D));
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) copy_to[(16 * m + 4 * n4 + r) * D + col] = S.s[m][r];
      }
    } else {
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) S.s[m][r] = identity && 16 * m + 4 * n4 + r == col ? 1.0f : 0.0f;
    }
    S.scale = S.inverse = 1.0f;
    S.apply(S.factor(column_max(S.largest())));
    most = S.largest();
  }

  const f16x8* const kq = (const f16x8*)krows;
  const f16x8* const qq = (const f16x8*)qrows;
  const f16x8* const kt = (const f16x8*)rest;
  const float* const factors = (const float*)(rest + kMatrix);
  const f16x8* const tp = (const f16x8*)(rest + kMatrix + 1024);
  const f16x8* const ap = (const f16x8*)(rest + kMatrix + 1024 + 6144);

  // Loads to LDS are counted per wave: each waits for its own before a barrier that lets the
  // others read.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  if (kParts == 1 && identity && begin == 0) {
    // Nobody needs the first segment's M: these waves only load.
    for (int left = end; left > 0; --left) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      slot += slot_step;
      if (left > 1) load_rows(slot);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (left > 1) load_rest(slot);
    }
    return;
  }

  for (int chunk = begin; chunk < end; ++chunk) {
    const int64_t first = seq.start + chunk * kChunk;
    const int valid = seq.len - chunk * kChunk < kChunk ? seq.len - chunk * kChunk : kChunk;
    typename Pair<kF>::raw rv[8];  // values: rows 16 t + 4 (lane / 16) + r, this lane's columns
    if (!identity) {
      const Window wv(R.v + (first * R.v_ts + h * R.v_hs) * kEB, valid, (uint32_t)R.v_ts * kEB, D * kEB);
      const uint32_t at = fresh(n4) * (4 * wv.stride) + col * kEB;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        rv[i] = Cell<kF>::one(wv, at, 16 * (i / 4) + i % 4);
      }
    }

    // ---- Y = (K e^G) S and O = (Q e^G) S
    f32x4 Y[2], O[2];
    Y[0] = Y[1] = O[0] = O[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // Steps of (32 channels, 16 rows). A step's left operands are read while the step before
    // runs; the scheduling barriers keep the steps apart.
    f16x8 kh, kl, qh, ql;
    const auto read_step = [&](int step) {
      const int kk = step >> 1, at = step * 128 + 16 * n4 + (n16 ^ (n4 + 4 * kk));
      kh = kq[at];
      kl = kq[at + 64];
      if (kOut) {
        qh = qq[at];
        ql = qq[at + 64];
      }
    };
    read_step(0);
    Operand b;
#pragma unroll
    for (int step = 0; step < 2 * kK; ++step) {
      const int t = step & 1;
      const f16x8 ch = kh, cl = kl, dh = qh, dl = ql;
      if (step + 1 < 2 * kK) read_step(step + 1);
      if (t == 0) b = split8(S.s[step], S.s[step + 1], R.one);
      Y[t] = mfma16(ch, b.hi, Y[t]);
      if (kOut) O[t] = mfma16(dh, b.hi, O[t]);
      Y[t] = mfma16(ch, b.lo, Y[t]);
      if (kOut) O[t] = mfma16(dh, b.lo, O[t]);
      Y[t] = mfma16(cl, b.hi, Y[t]);
      if (kOut) O[t] = mfma16(dl, b.hi, O[t]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // This chunk's other operands and values have arrived, and all waves are done with its
    // rows. (Said of the values too: the compiler would wait for them at their use, and so
    // for the loads issued until then.)
    asm volatile("s_waitcnt vmcnt(0)"
                 : "+v"(rv[0]), "+v"(rv[1]), "+v"(rv[2]), "+v"(rv[3]), "+v"(rv[4]), "+v"(rv[5]),
                   "+v"(rv[6]), "+v"(rv[7])
                 :
                 : "memory");
    __syncthreads();
    slot += slot_step;

    // ---- X = V - n Y, in the columns' scales
    if (identity || valid != kChunk) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (identity || 16 * (i / 4) + 4 * n4 + i % 4 >= valid) rv[i] = Pair<kF>::zero();
    }
    f32x4 X[2];
    const auto difference = [&]() {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f32x4 nt = *(const f32x4*)(factors + kFactorRows + 16 * t + 4 * n4);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          X[t][r] = __builtin_fmaf(Pair<kF>::value(rv[4 * t + r]).x, S.scale, -nt[r] * Y[t][r]);
      }
    };
    // What the column's values are measured by beside X and U: S, unless this chunk empties it.
    // Then what X and U hold is all that is left, however far below S it is.
    float beside = factors[kFactorFaded] != 0.0f ? most : 0.0f;
    // The column's range over X, NaN where an X is.
    const auto range = [&](float m) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = __builtin_elementwise_maximum(m, __builtin_fabsf(X[t][r]));
      return m;
    };
    float back = 1.0f;  // what X was divided by
    difference();
    float high = range(beside);
    if (!S.within(high) || S.below(high)) {
      // Values beyond a faded column's scale: that goes back to 1 first.
      bool beyond = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) beyond |= __builtin_fabsf(X[i / 4][i % 4]) == __builtin_huge_valf();
      if (column_max(beyond ? 1.0f : 0.0f) != 0.0f && S.scale > 1.0f) {
        const float f = S.inverse;
        S.apply(f);
        beside *= f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          Y[t] *= f;
          O[t] *= f;
        }
        difference();
      }
      // An X that is still not finite would reach all rows of its column (T's zeros times NaN).
      // By the definition it reaches those from its own on: they are left out of the products
      // here, and start O, and S, from NaN.
      int dead = kChunk;  // the column's first such row
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (!is_finite(X[i / 4][i % 4])) dead = 16 * (i / 4) + 4 * n4 + i % 4;
      if (__ballot(dead < kChunk) != 0) {
        int other = __shfl_xor(dead, 16);
        dead = dead < other ? dead : other;
        other = __shfl_xor(dead, 32);
        dead = dead < other ? dead : other;
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * (i / 4) + 4 * n4 + i % 4 >= dead) {
            X[i / 4][i % 4] = 0.0f;
            O[i / 4][i % 4] = nan;
          }
        if (dead < kChunk) {
#pragma unroll
          for (int m = 0; m < kM; ++m) S.s[m] = f32x4{nan, nan, nan, nan};
        }
      }
      // X alone, for its product with T: the U that comes of it may be far smaller (steps near
      // 0, short keys).
      const float m = column_max(range(0.0f));
      if (m > 0.0f && (m >= kColHigh || m < kColLow)) {
        int e = kColExp - __builtin_amdgcn_frexp_expf(m);
        e = e < 100 ? e : 100;
        back = __builtin_amdgcn_ldexpf(1.0f, -e);
#pragma unroll
        for (int t = 0; t < 2; ++t) X[t] *= __builtin_amdgcn_ldexpf(1.0f, e);
      }
    }

    // ---- U = T X
    f32x4 U[2];
    b = split8(X[0], X[1], R.one);
    const float us = factors[kFactorT] * back;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const f16x8 th = tp[64 * t + lane], tl = tp[128 + 64 * t + lane], tr = tp[256 + 64 * t + lane];
      f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
      u = mfma16(tr, b.hi, u);
      u = mfma16(tl, b.hi, u);
      u = mfma16(th, b.lo, u);
      u = mfma16(th, b.hi, u);
      U[t] = u * us;
    }
    // (Issued here and not right after the barrier: the products with T then start 300 cycles
    // earlier, and the loads still have the rest of the chunk to arrive.)
    if (chunk + 1 < end) load_rows(slot);
    // The column's range over U and what S keeps: the larger of them keeps its bits.
    high = beside;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) high = __builtin_fmaxf(high, __builtin_fabsf(U[t][r]));
    if (!S.within(high) || S.below(high)) {
      const float f = S.factor(column_max(high));
      S.apply(f);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        U[t] *= f;
        O[t] *= f;
      }
    }

    // ---- S <- e^G_end S + K^T U; O += A U
    const Operand u = split8(U[0], U[1], R.one);
    f16x8 ah, al;
    f32x4 d;
    const auto read_tile = [&](int m) {
      d = *(const f32x4*)(factors + 16 * m + 4 * n4);
      ah = kt[128 * m + lane];
      al = kt[128 * m + 64 + lane];
    };
    read_tile(0);
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const f16x8 ch = ah, cl = al;
      const f32x4 e = d;
      if (m + 1 < kM) read_tile(m + 1);
      S.s[m] = mfma16(ch, u.hi, S.s[m] * e);
      S.s[m] = mfma16(ch, u.lo, S.s[m]);
      S.s[m] = mfma16(cl, u.hi, S.s[m]);
      if (m & 1) __builtin_amdgcn_sched_barrier(0);
    }
    if (kOut) {
      const Window wo(R.out + (first * R.heads + h) * (D * kEB), valid, (uint32_t)R.heads * (D * kEB), D * kEB);
      const uint32_t at = fresh(n4) * (4 * wo.stride) + col * kEB;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f16x8 ah = ap[64 * t + lane], al = ap[128 + 64 * t + lane];
        const f32x4 nq = *(const f32x4*)(factors + kFactorRows + kChunk + 16 * t + 4 * n4);
        O[t] = mfma16(ah, u.hi, O[t]);
        O[t] = mfma16(ah, u.lo, O[t]);
        O[t] = mfma16(al, u.hi, O[t]);
#pragma unroll
        for (int r = 0; r < 4; ++r) O[t][r] = O[t][r] * S.inverse * nq[r];  // (nq * inverse may be subnormal)
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) Cell<kF>::store_one(wo, at, 16 * (i / 4) + i % 4, O[i / 4][i % 4]);
    }
    // The column's range for the next chunk.
    most = S.largest();
    if (!S.within(most) || S.below(most)) {
      const float f = S.factor(column_max(most));
      S.apply(f);
      most *= f;
    }
    // The next chunk's rows have arrived, and all waves are done with this chunk.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (chunk + 1 < end) load_rest(slot);
  }

  // ---- the end
  if (!identity) {
    float* to = nullptr;
    if (!kOut)
      to = P.ends + cell * (D * D);
    else if (end == chunks && seq.line >= 0)
      to = R.states + seq.line * R.st_line + h * R.st_head;
    if (to != nullptr) {
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[(16 * m + 4 * n4 + r) * D + col] = S.s[m][r] * S.inverse;
    }
  }
  if (!kOut && begin > 0) {
    // M as pairs in operand order, scaled by one power of two to a largest entry of 256 to
    // 512.
    float top = 0.0f;
    if (identity) {
      S.apply(S.inverse);
      top = S.largest();
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, m));
      if (lane == 0) part[cw] = top;
    }
    __syncthreads();
    if (identity) {
#pragma unroll
      for (int w = 0; w < kColWaves; ++w) top = __builtin_fmaxf(top, part[w]);
      int e = 0;
      if (top > 0.0f && top < __builtin_huge_valf()) e = 9 - __builtin_amdgcn_frexp_expf(top);
      e = e > 100 ? 100 : e;
      char* const to = P.moves + cell * move_bytes(D);
      _Float16* const hi = (_Float16*)to;
      const int pl = place(col % 32);
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = __builtin_amdgcn_ldexpf(S.s[m][r], e);
          const int at = ((m * kK + col / 32) * 64 + (pl / 8) * 16 + 4 * n4 + r) * 8 + pl % 8;
          hi[at] = (_Float16)x;
          hi[D * D + at] = (_Float16)(x - (float)(_Float16)x);
        }
      if (cw == 0 && lane == 0) *(float*)(to + (int64_t)D * D * 4) = __builtin_amdgcn_ldexpf(1.0f, -e);
    }
  }
}

// ------------------------------------------------------------------------------- join

// The starts of a sequence's segments: ends[0] is segment 0's end and so segment 1's
// start; ends[j] <- M_j ends[j - 1] + ends[j] makes it segment j + 1's start. One workgroup
// per (sequence, head, 16 columns); wave w owns rows 16 w .. of the columns and hands its
// operands to the others through LDS. A step is short, so M and B are loaded kAhead steps
// ahead. Workgroups of one (sequence, head) read the same M: the grid's rows are whole
// multiples of 8, which puts them on one of the card's 8 dies and in one L2.
//
// A step takes 1.3 us (1.6 with its loads issued at once): the 64 KB of M alone are 0.5 at a
// CU's 64 bytes per cycle, the rest is the chain largest value - split - exchange - product.
// Fewer, longer segments make it shorter, not more workgroups.
template <int D>
__global__ __launch_bounds__(4 * D, 2) void delta_rule_join_kernel(const ChunkParams P) {
  constexpr int kK = D / 32, kWaves = D / 16, kAhead = 2;
  __shared__ __attribute__((aligned(16))) _Float16 hi[2][kK][64 * 8], lo[2][kK][64 * 8];
  __shared__ float most[2][kWaves][16];
  const RuleParams& R = P.R;
  const int program = blockIdx.x / R.heads, h = blockIdx.x % R.heads, slice = blockIdx.y;
  const int wave = uniform(threadIdx.x / kRuleWave), lane = threadIdx.x % kRuleWave;
  if (program >= P.join_programs) return;
  const Piece piece = find_piece(P, P.join_pieces, program, lane);
  if (piece.s < 0 || piece.index != 0) return;
  const Sequence seq(R, piece.s);
  if (seq.len < P.min_len) return;
  const int chunks = (seq.len + kChunk - 1) / kChunk;
  const int per = chunks_per_segment(P, chunks);
  const int segments = (chunks + per - 1) / per;
  if (segments < 3) return;
  const int n16 = lane % 16, n4 = lane / 16;
  const int64_t cell = (int64_t)P.move_pieces.first(piece.s, seq.start) * R.heads + h;
  float* const ends = P.ends + cell * (D * D) + (16 * wave + 4 * n4) * D + 16 * slice + n16;
  const char* const moves = P.moves + cell * move_bytes(D);

  // A step's M rows and B.
  struct Step {
    f16x8 ah[kK], al[kK];
    float back;
    f32x4 B;
  };
  // In three parts: half of M's rows each, and B. A workgroup's loads of a step keep the CU's
  // address unit busy for 1300 cycles, so they are issued where the waves wait for each other.
  const auto load = [&](int j, Step& x, int part) {
    j = j < segments - 1 ? j : segments - 2;
    const char* const move = moves + (int64_t)j * R.heads * move_bytes(D);
    if (part < 2) {
      const f16x8* const a = (const f16x8*)move + wave * kK * 64 + lane;
#pragma unroll
      for (int kk = 0; kk < kK / 2; ++kk) {
        const int k = part * (kK / 2) + kk;
        x.ah[k] = a[64 * k];
        x.al[k] = a[64 * k + D * D / 8];
      }
    } else {
      x.back = *(const float*)(move + (int64_t)D * D * 4);
      const float* const end = ends + (int64_t)j * R.heads * (D * D);
#pragma unroll
      for (int r = 0; r < 4; ++r) x.B[r] = end[r * D];
    }
  };
  f32x4 S;
#pragma unroll
  for (int r = 0; r < 4; ++r) S[r] = ends[r * D];
  const auto step = [&](int j, const Step& x, Step& ahead) {
    const int buf = j & 1;
    float m = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(S[0]), __builtin_fabsf(S[1])),
                              __builtin_fmaxf(__builtin_fabsf(S[2]), __builtin_fabsf(S[3])));
    m = column_max(m);
    if (n4 == 0) most[buf][wave][n16] = m;
    load(j + kAhead, ahead, 0);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = __builtin_fmaxf(m, most[buf][w][n16]);
    int e = 0;
    if (m > 0.0f && m < __builtin_huge_valf()) e = kColExp - __builtin_amdgcn_frexp_expf(m);
    e = e > 100 ? 100 : e;
    {
      f32x4 s;
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = __builtin_amdgcn_ldexpf(S[r], e);
      const HalfPair p0 = split2(f32x2{s[0], s[1]}, R.one), p1 = split2(f32x2{s[2], s[3]}, R.one);
      const int at = lane * 8 + 4 * (wave & 1);
      *(f16x4*)&hi[buf][wave / 2][at] = f16x4{p0.hi.x, p0.hi.y, p1.hi.x, p1.hi.y};
      *(f16x4*)&lo[buf][wave / 2][at] = f16x4{p0.lo.x, p0.lo.y, p1.lo.x, p1.lo.y};
    }
    load(j + kAhead, ahead, 1);
    __syncthreads();
    const float f = __builtin_amdgcn_ldexpf(x.back, -e);
    f32x4 hh = {0.0f, 0.0f, 0.0f, 0.0f}, hl = hh, lh = hh;
#pragma unroll
    for (int kk = 0; kk < kK; ++kk) {
      const f16x8 bh = *(const f16x8*)&hi[buf][kk][lane * 8], bl = *(const f16x8*)&lo[buf][kk][lane * 8];
      hh = mfma16(x.ah[kk], bh, hh);
      hl = mfma16(x.ah[kk], bl, hl);
      lh = mfma16(x.al[kk], bh, lh);
    }
    load(j + kAhead, ahead, 2);
    hh += hl + lh;
    float* const end = ends + (int64_t)j * R.heads * (D * D);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      S[r] = __builtin_fmaf(hh[r], f, x.B[r]);
      end[r * D] = S[r];
    }
  };
  // Left from the middle: a condition around each step made the compiler move the loaded
  // registers at its end, and so wait for them.
  Step x[kAhead + 1];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int part = 0; part < 3; ++part) load(1 + i, x[i], part);
  for (int j = 1;;) {
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) {
      step(j, x[i], x[(i + kAhead) % (kAhead + 1)]);
      if (++j == segments - 1) return;
    }
  }
}

// ----------------------------------------------------------------------------- launches

template <int kF, int kG, int D>
void launch_chunks(const ChunkParams& P, hipStream_t st) {
  const unsigned heads = (unsigned)P.R.heads;
  const unsigned chunks = (unsigned)P.chunk_programs * heads;
  const unsigned segments = (unsigned)P.segment_programs * heads;
  const unsigned moves = (unsigned)P.move_programs * heads, joins = (unsigned)P.join_programs * heads;
  if (D == 128 && P.wide)
    hipLaunchKernelGGL((delta_rule_prepare_kernel<kF, kG, D, D / 16>), dim3(chunks), dim3(4 * D), 0, st, P);
  else
    hipLaunchKernelGGL((delta_rule_prepare_kernel<kF, kG, D, 4>), dim3(chunks), dim3(256), 0, st, P);
  if (P.moves != nullptr) {
    // Two workgroups per segment and head, one for B and one for M, where that makes at most two
    // per CU: each CU then reads half as many operands from LDS (60 segments of 4 chunks 22.4 us
    // against 17.3, 192 28.9 against 28.0; the operands are loaded twice).
    if (moves <= 256)
      hipLaunchKernelGGL((delta_rule_scan_kernel<kF, D, kScanMove, 2>), dim3(moves, 2), dim3(4 * D), 0, st, P);
    else
      hipLaunchKernelGGL((delta_rule_scan_kernel<kF, D, kScanMove, 1>), dim3(moves), dim3(8 * D), 0, st, P);
    hipLaunchKernelGGL((delta_rule_join_kernel<D>), dim3((joins + 7) / 8 * 8, D / 16), dim3(4 * D), 0, st, P);
  }
  hipLaunchKernelGGL((delta_rule_scan_kernel<kF, D, kScanOut, 1>), dim3(segments), dim3(4 * D), 0, st, P);
}

template <int kF, int kG>
void launch_rule_chunks(const ChunkParams& P, int head_dim, hipStream_t st) {
  if (head_dim == 128)
    launch_chunks<kF, kG, 128>(P, st);
  else
    launch_chunks<kF, kG, 64>(P, st);
}

}  // namespace kdaconv

#endif  // KDACONV_DELTA_RULE_CHUNK_H_
