// The gated delta rule: checks of arguments and the C entry points. include/kdaconv.h
// states the operator.
#include "delta_rule.h"

#include <algorithm>
#include <initializer_list>

namespace kdaconv {
namespace {

// 32 rows stay below 2^30 bytes.
constexpr int64_t kMaxStride = (int64_t)1 << 23;

bool known_rule_dtype(int d) { return d == KDACONV_BF16 || d == KDACONV_F16 || d == KDACONV_F32; }

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

int64_t dtype_size(int d) { return d == KDACONV_F32 ? 4 : 2; }

// How a prefill call is worked on. It depends on host sizes alone.
struct Plan {
  bool step;  // the step kernel takes sequences of up to max_len tokens
  bool chunks;  // the chunked kernels take the others
  bool segments;  // sequences of several segments are possible
  bool wide;  // prepare takes 8 waves per chunk of 128 channels
  int64_t max_len;
  int segment_chunks;
  int whole_chunks;  // sequences of up to so many are not cut
  Pieces chunk_pieces, segment_pieces, move_pieces, join_pieces;
  int64_t chunk_programs, segment_programs, move_programs, join_programs;
  int64_t slot_bytes, ends_bytes, moves_bytes;
};

// Sequences of up to this many tokens are faster token by token. (12 heads of 128: one
// sequence of 12 tokens takes 24 us against 29 in a chunk, one of 24 41 against 30; 256
// sequences of 12 tokens 161 against 236, of 24 261 against 246.)
constexpr int64_t kStepTokens = 16;
// The step kernel is launched beside the chunked ones, which then leave those sequences out,
// where sequences average up to kStepAverage tokens, or under kStepAverageMany and make
// kStepMany workgroups. (Every sequence of 4 tokens: 32 of 12 heads take 24 us against 42 by
// chunks alone, 256 take 105 against 224. Lengths uniform about 24 tokens: 64 sequences 107
// against 91, 256 266 against 276. About 20, 30 sequences of 4 heads: 61 against 36.)
constexpr int64_t kStepAverage = 8, kStepAverageMany = 32, kStepMany = 2048;
// Segments: as long as leaves one for each of this many CUs, and no shorter than kSegmentMin
// chunks. A segment that is not a sequence's last is worked on twice, at twice the columns;
// but where the sequences alone make more than two workgroups per CU the longest of them are
// what a call waits for, and segments are shorter by a third. (16384 tokens of 12 heads: one
// sequence 449 us, with half as long segments 499; 64 prompts of log-normal lengths, over 12
// draws, 376 us on average and 401 at most, with segments three times as long 420 and 526,
// though prompts of uniform lengths take 326 and 306. 24 log-normal prompts: 400, with twice
// as long segments 518. 3 sequences of 2999 tokens in all, 8 heads, 106 us, segments of 3
// chunks 121; 8 prompts of 1204 tokens, 12 heads, 77, segments of 6 chunks 81.)
constexpr int64_t kSegmentCells = 256, kSegmentMin = 4;
// Sequences of up to kWhole chunks stay whole where they are likely all that short: one that is,
// or several of half that on average. (8 prompts of 1204 tokens, 12 heads: 69 us against 78;
// one of 320 tokens 49 against 59, the launches that only cut ones need left out. But a
// call waits for its longest whole sequence and for its cut ones: 8 prompts of 2400 tokens
// would take 116 us, not 108, 3 sequences of 2999 tokens 104, not 101.)
constexpr int64_t kWhole = 12;
// Chunks get 8 waves in prepare where about this many workgroups, two per CU, are all there
// are, else 4. A sequence's last chunk is counted half: some have none. (2 chunks 10.7 us
// against 11.6, 500 19 against 22; 650 26 against 23, 6144 170 against 142.)
constexpr int64_t kWideCells = 512;

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

Plan make_plan(int64_t tokens, int64_t seqs, int64_t heads, int64_t head_dim) {
  Plan p = {};
  p.step = tokens <= kStepTokens || tokens <= kStepAverage * seqs ||
           (tokens < kStepAverageMany * seqs && seqs * heads >= kStepMany);
  p.chunks = tokens > kStepTokens;
  p.max_len = p.step ? kStepTokens : 0;
  const int64_t cells = seqs * heads > 2 * kSegmentCells ? kSegmentCells * 3 / 2 : kSegmentCells;
  const int64_t units = (tokens + kChunk - 1) / kChunk * heads;
  p.segment_chunks = (int)std::max(kSegmentMin, (units + cells - 1) / cells);
  const int64_t segment = (int64_t)p.segment_chunks * kChunk;
  p.wide = (tokens / kChunk + (seqs + 1) / 2) * heads <= kWideCells;
  p.whole_chunks = tokens * (seqs > 1 ? 2 : 1) <= kWhole * kChunk * seqs ? (int)kWhole : 0;
  p.segments = tokens > std::max(segment, (int64_t)p.whole_chunks * kChunk);
  const auto pieces = [&](int64_t piece_tokens, Pieces& how) {
    const int64_t all = tokens / piece_tokens + seqs;
    // Sequences of more than max_len tokens alone: max_len tokens and more per program are
    // enough for a piece of 32 or more.
    const int64_t longer = p.max_len > 0 ? tokens / p.max_len + 1 : all;
    how = longer < all ? Pieces{(int32_t)p.max_len, 0} : Pieces{(int32_t)piece_tokens, 1};
    return std::min(all, longer);
  };
  p.chunk_programs = pieces(kChunk, p.chunk_pieces);
  p.segment_programs = pieces(segment, p.segment_pieces);
  // Of n tokens ceil(n / segment) - 1 <= floor(n / segment) segments are not the last.
  p.move_pieces = Pieces{(int32_t)segment, 0};
  p.move_programs = tokens / segment + 1;
  p.join_pieces = Pieces{(int32_t)(2 * segment), 0};
  p.join_programs = tokens / (2 * segment) + 1;
  if (p.chunks) {
    p.slot_bytes = round256(p.chunk_programs * heads * Slot{head_dim}.bytes());
    if (p.segments) {
      p.ends_bytes = round256(p.move_programs * heads * head_dim * head_dim * 4);
      p.moves_bytes = p.move_programs * heads * move_bytes((int)head_dim);
    }
  }
  return p;
}

// Workgroups of the largest launch, of up to 512 threads: a launch may not reach 2^32 threads.
// (The transitions' have 1024, but moves and joins are at most 3/2 kSegmentCells + heads.)
constexpr int64_t kMaxGrid = (int64_t)1 << 23;

int64_t largest_grid(const kdaconv_rule_args* a, bool update) {
  const int64_t heads = std::max<int64_t>(1, a->num_heads), steps = a->num_seqs * heads;
  if (update) return steps;
  const Plan p = make_plan(a->num_tokens, a->num_seqs, heads, a->head_dim);
  return std::max(p.step ? steps : 0, p.chunks ? std::max(p.chunk_programs, p.segment_programs) * heads : 0);
}

int validate_rule(const kdaconv_rule_args* a, bool update) {
  if (a == nullptr) return KDACONV_EINVAL;
  if (a->num_tokens < 0 || a->num_seqs < 0 || a->num_heads < 0 || a->num_cache_lines < 0)
    return KDACONV_EINVAL;
  if (!known_rule_dtype(a->dtype) || !known_rule_dtype(a->gate_dtype) ||
      !known_rule_dtype(a->beta_dtype))
    return KDACONV_EINVAL;
  if (a->gate != KDACONV_GATE_LOG && a->gate != KDACONV_GATE_SOFTPLUS &&
      a->gate != KDACONV_GATE_BOUNDED)
    return KDACONV_EINVAL;
  if (a->head_dim <= 0 || a->num_qk_heads <= 0 || a->num_heads % a->num_qk_heads != 0)
    return KDACONV_EINVAL;
  if (a->g_stride2 != 0 && a->g_stride2 != 1) return KDACONV_EINVAL;
  if (update && a->num_tokens != a->num_seqs) return KDACONV_EINVAL;
  if (a->lower_bound > 0.0 || a->lower_bound != a->lower_bound) return KDACONV_EINVAL;
  if (a->head_dim != 64 && a->head_dim != 128) return KDACONV_EUNSUPPORTED;
  if (a->gate_dtype != a->dtype && a->gate_dtype != KDACONV_F32) return KDACONV_EUNSUPPORTED;
  if (a->beta_dtype != a->dtype && a->beta_dtype != KDACONV_F32) return KDACONV_EUNSUPPORTED;
  // (The stride of an axis of one means nothing.)
  const struct {
    int64_t count;
    std::initializer_list<int64_t> strides;
  } axes[] = {{a->num_tokens, {a->q_stride0, a->k_stride0, a->v_stride0, a->g_stride0, a->beta_stride0}},
              {a->num_qk_heads, {a->q_stride1, a->k_stride1}},
              {a->num_heads, {a->v_stride1, a->g_stride1, a->beta_stride1}}};
  for (const auto& axis : axes)
    for (int64_t s : axis.strides)
      if (axis.count != 1 && (s < 0 || s >= kMaxStride)) return KDACONV_EUNSUPPORTED;
  if (a->state_stride0 < 0 || a->state_stride1 < 0 || a->cache_indices_stride < 0)
    return KDACONV_EUNSUPPORTED;
  // int32 tokens, sequences and workgroups.
  if (a->num_tokens > INT32_MAX / 2 || a->num_seqs > INT32_MAX / 2 || a->num_heads > 65535)
    return KDACONV_EUNSUPPORTED;
  if ((a->num_tokens + a->num_seqs) * std::max<int64_t>(1, a->num_heads) > INT32_MAX / 4)
    return KDACONV_EUNSUPPORTED;
  if (largest_grid(a, update) >= kMaxGrid) return KDACONV_EUNSUPPORTED;
  if (a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0) return KDACONV_OK;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->states || !a->cache_indices || !a->out)
    return KDACONV_EINVAL;
  if (!update && !a->query_start_loc) return KDACONV_EINVAL;
  if (a->gate != KDACONV_GATE_LOG && !a->a_log) return KDACONV_EINVAL;
  const int64_t eb = dtype_size(a->dtype);
  if (!aligned_to(a->q, eb) || !aligned_to(a->k, eb) || !aligned_to(a->v, eb) ||
      !aligned_to(a->out, eb) || !aligned_to(a->g, dtype_size(a->gate_dtype)) ||
      !aligned_to(a->beta, dtype_size(a->beta_dtype)) || !aligned_to(a->states, 4) ||
      !aligned_to(a->a_log, 4) || !aligned_to(a->dt_bias, 4))
    return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

RuleParams rule_params(const kdaconv_rule_args* a, bool update) {
  RuleParams P;
  P.q = static_cast<const char*>(a->q);
  P.k = static_cast<const char*>(a->k);
  P.v = static_cast<const char*>(a->v);
  P.g = static_cast<const char*>(a->g);
  P.beta = static_cast<const char*>(a->beta);
  P.a_log = a->a_log;
  P.dt_bias = a->gate == KDACONV_GATE_LOG ? nullptr : a->dt_bias;
  P.states = a->states;
  P.qsl = update ? nullptr : a->query_start_loc;
  P.cache_indices = a->cache_indices;
  P.has_init = update ? nullptr : a->has_initial_state;
  P.out = static_cast<char*>(a->out);
  const int64_t tokens = a->num_tokens != 1, qk_heads = a->num_qk_heads != 1, heads = a->num_heads != 1;
  P.q_ts = a->q_stride0 * tokens;
  P.q_hs = a->q_stride1 * qk_heads;
  P.k_ts = a->k_stride0 * tokens;
  P.k_hs = a->k_stride1 * qk_heads;
  P.v_ts = a->v_stride0 * tokens;
  P.v_hs = a->v_stride1 * heads;
  P.g_ts = a->g_stride0 * tokens;
  P.g_hs = a->g_stride1 * heads;
  P.g_cs = (int32_t)a->g_stride2;
  P.b_ts = a->beta_stride0 * tokens;
  P.b_hs = a->beta_stride1 * heads;
  P.st_line = a->state_stride0;
  P.st_head = a->state_stride1;
  P.num_cache_lines = a->num_cache_lines;
  P.ci_stride = a->cache_indices_stride;
  P.null_block_id = a->null_block_id;
  P.scale = (float)a->scale;
  P.l2_eps = (float)a->l2_eps;
  P.lower_bound = (float)a->lower_bound;
  P.num_tokens = (int32_t)a->num_tokens;
  P.num_seqs = (int32_t)a->num_seqs;
  P.heads = (int32_t)a->num_heads;
  P.share = (int32_t)(a->num_heads / a->num_qk_heads);
  P.gate = a->gate;
  P.beta_logits = a->beta_logits != 0;
  P.beta_f32 = a->beta_dtype == KDACONV_F32;
  P.has_null_block = a->has_null_block != 0;
  P.all_init = update;
  P.max_len = INT32_MAX;
  P.one = 1.0f;
  return P;
}

// Calls op.template run<x format, gate format>() for the call's formats.
template <class Op>
void for_formats(const kdaconv_rule_args* a, Op op) {
  if (a->dtype == KDACONV_F32)
    op.template run<KDACONV_F32, KDACONV_F32>();
  else if (a->dtype == KDACONV_F16 && a->gate_dtype == KDACONV_F32)
    op.template run<KDACONV_F16, KDACONV_F32>();
  else if (a->dtype == KDACONV_F16)
    op.template run<KDACONV_F16, KDACONV_F16>();
  else if (a->gate_dtype == KDACONV_F32)
    op.template run<KDACONV_BF16, KDACONV_F32>();
  else
    op.template run<KDACONV_BF16, KDACONV_BF16>();
}

struct Step {
  const RuleParams& P;
  int head_dim;
  hipStream_t st;
  template <int kF, int kG>
  void run() {
    launch_rule_step<kF, kG>(P, head_dim, st);
  }
};

struct Chunks {
  const ChunkParams& P;
  int head_dim;
  hipStream_t st;
  template <int kF, int kG>
  void run() {
    launch_rule_chunks<kF, kG>(P, head_dim, st);
  }
};

bool nothing(const kdaconv_rule_args* a) {
  return a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0;
}

}  // namespace
}  // namespace kdaconv

using namespace kdaconv;

extern "C" int64_t kdaconv_gated_delta_rule_workspace(int64_t num_tokens, int64_t num_seqs,
                                                      int64_t num_heads, int64_t head_dim) {
  if (num_tokens <= 0 || num_seqs <= 0 || num_heads <= 0 || head_dim <= 0) return 0;
  const Plan p = make_plan(num_tokens, num_seqs, num_heads, head_dim);
  return p.slot_bytes + p.ends_bytes + p.moves_bytes;
}

extern "C" int kdaconv_gated_delta_rule_validate(const kdaconv_rule_args* args, int update,
                                                 const void* workspace, int64_t workspace_bytes) {
  const int rc = validate_rule(args, update != 0);
  if (rc != KDACONV_OK || update != 0 || nothing(args)) return rc;
  const int64_t need = kdaconv_gated_delta_rule_workspace(args->num_tokens, args->num_seqs,
                                                          args->num_heads, args->head_dim);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KDACONV_EINVAL;
  if (need > 0 && !aligned_to(workspace, 256)) return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

extern "C" int kdaconv_gated_delta_rule(const kdaconv_rule_args* args, void* workspace,
                                        int64_t workspace_bytes, kdaconv_stream_t stream) {
  const int rc = kdaconv_gated_delta_rule_validate(args, 0, workspace, workspace_bytes);
  if (rc != KDACONV_OK || nothing(args)) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const Plan plan = make_plan(args->num_tokens, args->num_seqs, args->num_heads, args->head_dim);
  ChunkParams P;
  P.R = rule_params(args, false);
  if (plan.step) {
    if (plan.chunks) P.R.max_len = (int32_t)plan.max_len;
    for_formats(args, Step{P.R, (int)args->head_dim, st});
  }
  if (plan.chunks) {
    P.slots = static_cast<char*>(workspace);
    P.ends = reinterpret_cast<float*>(P.slots + plan.slot_bytes);
    P.moves = plan.segments ? P.slots + plan.slot_bytes + plan.ends_bytes : nullptr;
    P.chunk_programs = (int32_t)plan.chunk_programs;
    P.segment_programs = (int32_t)plan.segment_programs;
    P.move_programs = (int32_t)plan.move_programs;
    P.join_programs = (int32_t)plan.join_programs;
    P.chunk_pieces = plan.chunk_pieces;
    P.segment_pieces = plan.segment_pieces;
    P.move_pieces = plan.move_pieces;
    P.join_pieces = plan.join_pieces;
    P.segment_chunks = plan.segment_chunks;
    P.whole_chunks = plan.whole_chunks;
    int64_t reach = kRuleWave;
    while (reach < args->num_seqs) reach *= kRuleWave;
    P.search_top = (int32_t)(reach / kRuleWave);
    P.min_len = (int32_t)plan.max_len + 1;
    P.wide = plan.wide;
    for_formats(args, Chunks{P, (int)args->head_dim, st});
  }
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}

extern "C" int kdaconv_gated_delta_rule_update(const kdaconv_rule_args* args,
                                               kdaconv_stream_t stream) {
  const int rc = validate_rule(args, true);
  if (rc != KDACONV_OK || nothing(args)) return rc;
  const RuleParams P = rule_params(args, true);
  for_formats(args, Step{P, (int)args->head_dim, reinterpret_cast<hipStream_t>(stream)});
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}
