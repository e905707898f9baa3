// Absorbed latent attention over the paged cache: parameters, and how a call is split.
#ifndef KDACONV_LATENT_ATTENTION_H_
#define KDACONV_LATENT_ATTENTION_H_

#include "latent.h"

namespace kdaconv {

// A block of rows that several workers share: the first of them and their number (0: none),
// and which block of which sequence.
struct Shared {
  int32_t first, count, s, b;
};

struct AttendParams {
  CacheView C;
  PageTable T;
  const char* ql;
  const char* qr;
  char* out;  // (tokens, heads, latent), contiguous
  const int32_t* seq_lens;
  const int32_t* qsl;  // null: sequence s owns row s
  float* partial;  // per slot kRows x latent sums, see Partial
  Shared* shared;  // per worker: the block that its part begins inside, and the one it ends inside
  int64_t ql_ts, ql_hs, qr_ts, qr_hs;  // bytes
  int32_t tokens, seqs, workers;
  int32_t most_keys;  // the table's width in keys, up to kMostKeys
  int32_t shift;
  Divider heads;
  float scale;  // times log2(e)
};

// A call's work is a line of units: for every sequence, for every block of its rows (a row is a
// head of a token), kBlockUnits for the block itself and one for each step of keys (2^shift
// steps, which keeps the line below 2^31 units). The workers (workgroups, one per CU) take equal
// parts of the line. They work it out for themselves from the lengths on the device, so that a
// captured call serves any lengths.
constexpr int kBlockUnits = 2;
// A part is no shorter than this (unless the line is). One sequence of 16000 keys, 502 units, in us:
// parts of 2 units and more 26.7, 3 23.7, 4 25.4, 6 25.5 (the join's reads against the longest part).
constexpr int kLeastUnits = 3;
constexpr int kWorkers = 256;

constexpr int kAttendWaves = 8;
// Blocks of 16 rows per workgroup, and how it takes keys: a step's keys lie in LDS while
// kRing - 1 more steps are under way. Few rows leave memory the time that products need not:
// short steps, many under way. More rows share longer steps. (LDS holds 4 steps of 32 keys, or 2
// of 64 beside the weights.)
constexpr int step_keys(int blocks) { return blocks == 4 ? 64 : 32; }
constexpr int ring_steps(int blocks) { return blocks == 4 ? 2 : 4; }  // powers of 2 up to 4
constexpr int kMostKeys = 1 << 30;  // of a sequence

// A block that several workers share leaves each one's sums in scratch memory, two slots a
// worker: slot 2 w of the part that ends a block, 2 w + 1 of one that does not.
struct Partial {
  int rows, latent;
  __host__ __device__ constexpr int64_t floats() const { return (int64_t)rows * (latent + 2); }
  // Sums, then each row's exponent and weight.
  __host__ __device__ constexpr int64_t exponent() const { return (int64_t)rows * latent; }
  __host__ __device__ constexpr int64_t weight() const { return (int64_t)rows * (latent + 1); }
};

// kQ: blocks of 16 rows per workgroup, 1, 2 or 4.
template <int kF, int kLatent, int kQ, bool kE4m3>
void launch_attend(const AttendParams& P, hipStream_t st);

}  // namespace kdaconv

#endif  // KDACONV_LATENT_ATTENTION_H_
