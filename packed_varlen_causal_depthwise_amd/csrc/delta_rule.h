// The gated delta rule: parameters shared by the host code and the kernels.
#ifndef KDACONV_DELTA_RULE_H_
#define KDACONV_DELTA_RULE_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kdaconv.h"

namespace kdaconv {

constexpr int kRuleWave = 64;

// One call of the rule. Strides are in elements and bounded by the host checks (a token
// stride below 2^23), so offsets inside a chunk fit 32 bits.
struct RuleParams {
  const char* q;
  const char* k;
  const char* v;
  const char* g;
  const char* beta;
  const float* a_log;
  const float* dt_bias;
  float* states;
  const int32_t* qsl;  // null: sequence s owns row s
  const int32_t* cache_indices;
  const uint8_t* has_init;
  char* out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, g_ts, g_hs, b_ts, b_hs;
  int64_t st_line, st_head;
  int64_t num_cache_lines;
  int64_t ci_stride;
  int64_t null_block_id;
  float scale, l2_eps, lower_bound;
  int32_t num_tokens, num_seqs, heads, share;  // share: value heads per query and key head
  int32_t g_cs;  // 1, or 0: one gate per head
  int32_t gate, beta_logits, beta_f32, has_null_block;
  int32_t all_init;  // every sequence starts from its line (the update)
  int32_t max_len;  // the step kernel leaves longer sequences alone
  float one;  // 1
};

constexpr int kChunk = 32;  // tokens per chunk

// How pieces of sequences are numbered: sequence s owns programs v(s) up to v(s + 1), where
// v(s) = s * extra + floor(start of s / tokens). With `extra` 1 that is at least
// ceil(n / tokens) programs for any n tokens, with `extra` 0 at least floor(n / tokens), and
// then none for most shorter sequences. Either way the number of programs needs no lengths.
struct Pieces {
  int32_t tokens, extra;
  __host__ __device__ int32_t first(int32_t s, int64_t start) const {
    return s * extra + (int32_t)((uint32_t)start / (uint32_t)tokens);
  }
};

// What the chunked kernels need beside the call: where chunks and segments lie, and the
// scratch memory.
struct ChunkParams {
  RuleParams R;
  char* slots;  // a Slot per (chunk program, head)
  float* ends;  // head_dim^2 per (move program, head): a segment's end, then the next's start
  // move_bytes per (move program, head): the segment's transition; of a sequence's first
  // segment a copy of the state that it starts from.
  char* moves;
  // Chunks; segments; segments but a sequence's last; sequences of 3 segments and more.
  int32_t chunk_programs, segment_programs, move_programs, join_programs;
  Pieces chunk_pieces, segment_pieces, move_pieces, join_pieces;
  int32_t segment_chunks, whole_chunks;  // chunks per segment; sequences of up to so many stay whole
  int32_t search_top;  // 64^(levels - 1), 64^levels >= num_seqs
  int32_t min_len;  // shorter sequences are left to the step kernel
  bool wide;  // 8 waves per chunk of 128 channels, not 4
};

// One chunk of one head as the scans read it, in pieces of 1 KB that are one matrix operand
// each (64 lanes x 8 FP16): K e^G, Q e^G and K e^(G_end - G) as pairs, decays and row
// factors, T as three parts, A as a pair.
struct Slot {
  int64_t head_dim;
  __host__ __device__ constexpr int64_t matrix() const { return 128 * head_dim; }  // a pair of 32 x head_dim
  __host__ __device__ constexpr int64_t kg() const { return 0; }
  __host__ __device__ constexpr int64_t qg() const { return matrix(); }
  __host__ __device__ constexpr int64_t kt() const { return 2 * matrix(); }
  __host__ __device__ constexpr int64_t factors() const { return 3 * matrix(); }  // 1 KB
  __host__ __device__ constexpr int64_t t() const { return 3 * matrix() + 1024; }
  __host__ __device__ constexpr int64_t a() const { return t() + 6144; }
  __host__ __device__ constexpr int64_t bytes() const { return a() + 4096; }
};

// In a slot's factors: decays over the chunk (head_dim), then |k| / 16 and the outputs'
// factors / 16 (kChunk each), T's factor, and 0 if the chunk empties the state (1 if not).
constexpr int kFactorRows = 128, kFactorT = kFactorRows + 2 * kChunk, kFactorFaded = kFactorT + 1;

// The transition: pairs of FP16 matrices and a scale.
inline __host__ __device__ int64_t move_bytes(int head_dim) { return (int64_t)head_dim * head_dim * 4 + 256; }

// Launchers, one set per format (kF: x, kG: gate), defined where they are instantiated.
template <int kF, int kG>
void launch_rule_step(const RuleParams& P, int head_dim, hipStream_t st);

template <int kF, int kG>
void launch_rule_chunks(const ChunkParams& P, int head_dim, hipStream_t st);

}  // namespace kdaconv

#endif  // KDACONV_DELTA_RULE_H_
