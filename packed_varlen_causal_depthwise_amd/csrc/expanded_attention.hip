// Expanded attention: checks of arguments and the C entry point. include/kdaconv.h states the
// operator.
#include "expanded_attention.h"

#include <algorithm>
#include <cmath>

namespace kdaconv {
namespace {

// Keys' and values' rows are counted from a step's first in 32 bits, a row times a stride of up to 24
// bits in bytes.
constexpr int64_t kMaxTokenStride = (int64_t)1 << 23;

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int kCus = 256;

int64_t blocks_of(int64_t tokens, int64_t seqs, int waves) { return tokens / (kWaveRows * waves) + seqs; }

// Workgroups take 128 rows where these are no more blocks than CUs, or sequences are shorter; else
// 256, which read keys half as often, and so where every block has 2048 keys and more. 12 heads, in
// us with 256 and 128: 8 prompts of 200 rows 21.2 and 18.5, 16 of them 22.6 and 33.5; 4 of 512 rows
// 28.9 and 26.2, 16 of them 60 and 77; 20 of 64 rows 20.7 and 12.0; 3 of 300 rows over 5000 keys
// 78 and 93.
int waves_of(int64_t tokens, int64_t keys, int64_t seqs, int64_t heads) {
  const bool many = tokens >= 128 * seqs && blocks_of(tokens, seqs, 4) * heads > kCus;
  return many || (tokens >= 256 * seqs && keys >= 2048 * seqs) ? 8 : 4;
}

int64_t programs_of(int64_t tokens, int64_t keys, int64_t seqs, int64_t heads) {
  return blocks_of(tokens, seqs, waves_of(tokens, keys, seqs, heads));
}

// Parts of a block's keys: where blocks are fewer than half the CUs, as many as give each CU one, of
// kLeastSteps steps on average or more. 12 heads of 128 + 64 channels, in us, with and without:
// 1 row over 16000 keys 53 and 451, 300 over 8000 65 and 216, 128 of 2 sequences over 2200 26 and
// 42, over 1024 20.3 and 22.9. Twice as many parts as CUs: 78, 96, 26, 20.
constexpr int kLeastSteps = 4, kMostSplits = 64;
int splits_of(int64_t tokens, int64_t keys, int64_t seqs, int64_t heads) {
  if (tokens <= 0 || keys <= 0 || seqs <= 0 || heads <= 0) return 1;
  const int64_t fill = kCus / (programs_of(tokens, keys, seqs, heads) * heads), long_enough = keys / (seqs * kExpandKeys * kLeastSteps);
  return (int)std::max<int64_t>(1, std::min<int64_t>({fill, long_enough, kMostSplits}));
}

int validate_expanded(const kdaconv_expanded_args* a) {
  if (a == nullptr) return KDACONV_EINVAL;
  if (a->num_tokens < 0 || a->num_keys < 0 || a->num_seqs < 0 || a->num_heads < 0 || a->key_dim <= 0 ||
      a->rope_dim < 0 || a->value_dim <= 0 || std::isnan(a->scale))
    return KDACONV_EINVAL;
  if (a->dtype != KDACONV_BF16 && a->dtype != KDACONV_F16 && a->dtype != KDACONV_F32) return KDACONV_EINVAL;
  if (a->dtype == KDACONV_F32) return KDACONV_EUNSUPPORTED;
  if (a->key_dim % 8 != 0 || a->key_dim > 128 || a->value_dim % 8 != 0 || a->value_dim > 128 ||
      a->rope_dim % 8 != 0 || a->rope_dim > kRopeMax)
    return KDACONV_EUNSUPPORTED;
  // Strides of axes of one entry mean nothing. Keys and values move in pieces of 16 bytes.
  const bool tokens = a->num_tokens > 1, keys = a->num_keys > 1, heads = a->num_heads > 1;
  if ((tokens && a->q_stride0 < 0) || (heads && a->q_stride1 < 0)) return KDACONV_EUNSUPPORTED;
  const struct {
    bool counts;
    int64_t stride, limit;
  } axes[] = {{keys, a->k_stride0, kMaxTokenStride},  {heads, a->k_stride1, INT64_MAX},
              {keys, a->v_stride0, kMaxTokenStride},  {heads, a->v_stride1, INT64_MAX},
              {keys && a->rope_dim > 0, a->kr_stride0, kMaxTokenStride}};
  for (const auto& axis : axes)
    if (axis.counts && (axis.stride < 0 || axis.stride >= axis.limit || axis.stride % 8 != 0)) return KDACONV_EUNSUPPORTED;
  if (a->num_tokens > INT32_MAX / 4 || a->num_keys > INT32_MAX / 4 || a->num_seqs > INT32_MAX / 4 || a->num_heads > 65535)
    return KDACONV_EUNSUPPORTED;
  // 2^32 threads.
  if (programs_of(a->num_tokens, a->num_keys, a->num_seqs, a->num_heads) * a->num_heads >= (int64_t)1 << 23) return KDACONV_EUNSUPPORTED;
  if (a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0) return KDACONV_OK;
  if (!a->q || !a->out || !a->query_start_loc || !a->kv_start_loc) return KDACONV_EINVAL;
  if (a->num_keys > 0 && (!a->k || !a->v || (a->rope_dim > 0 && !a->k_rope))) return KDACONV_EINVAL;
  if (!aligned_to(a->q, 2) || !aligned_to(a->out, 2) || !aligned_to(a->k, 16) || !aligned_to(a->v, 16) ||
      (a->rope_dim > 0 && !aligned_to(a->k_rope, 16)) || !aligned_to(a->query_start_loc, 4) || !aligned_to(a->kv_start_loc, 4))
    return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

template <int kF, int kDim, int kRope>
void launch(const ExpandParams& P, int waves, hipStream_t st) {
  if (waves == 8)
    launch_expanded<kF, kDim, kRope, 8>(P, st);
  else
    launch_expanded<kF, kDim, kRope, 4>(P, st);
}

template <int kF>
void launch(const ExpandParams& P, bool wide, bool rope, int waves, hipStream_t st) {
  if (wide && rope)
    launch<kF, 128, 64>(P, waves, st);
  else if (wide)
    launch<kF, 128, 32>(P, waves, st);
  else if (rope)
    launch<kF, 64, 64>(P, waves, st);
  else
    launch<kF, 64, 32>(P, waves, st);
}

}  // namespace
}  // namespace kdaconv

using namespace kdaconv;

extern "C" int64_t kdaconv_expanded_attention_workspace(int64_t num_tokens, int64_t num_keys, int64_t num_seqs,
                                                        int64_t num_heads, int64_t value_dim) {
  const int splits = splits_of(num_tokens, num_keys, num_seqs, num_heads);
  if (splits == 1 || value_dim <= 0) return 0;
  const ExpandPartial part{kWaveRows * waves_of(num_tokens, num_keys, num_seqs, num_heads), (int)value_dim};
  return programs_of(num_tokens, num_keys, num_seqs, num_heads) * num_heads * splits * part.floats() * (int64_t)sizeof(float);
}

extern "C" int kdaconv_expanded_attention_validate(const kdaconv_expanded_args* args, const void* workspace,
                                                   int64_t workspace_bytes) {
  const int rc = validate_expanded(args);
  if (rc != KDACONV_OK) return rc;
  const int64_t need = kdaconv_expanded_attention_workspace(args->num_tokens, args->num_keys, args->num_seqs,
                                                            args->num_heads, args->value_dim);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KDACONV_EINVAL;
  if (need > 0 && !aligned_to(workspace, 256)) return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

extern "C" int kdaconv_expanded_attention(const kdaconv_expanded_args* a, void* workspace, int64_t workspace_bytes,
                                          kdaconv_stream_t stream) {
  const int rc = kdaconv_expanded_attention_validate(a, workspace, workspace_bytes);
  if (rc != KDACONV_OK || a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0) return rc;
  ExpandParams P;
  P.q = static_cast<const char*>(a->q);
  P.k = static_cast<const char*>(a->k);
  P.kr = static_cast<const char*>(a->k_rope);
  P.v = static_cast<const char*>(a->v);
  P.out = static_cast<char*>(a->out);
  P.qsl = a->query_start_loc;
  P.ksl = a->kv_start_loc;
  const int64_t tokens = a->num_tokens > 1, keys = a->num_keys > 1, heads = a->num_heads > 1;
  P.q_ts = a->q_stride0 * 2 * tokens;
  P.q_hs = a->q_stride1 * 2 * heads;
  P.k_ts = a->k_stride0 * 2 * keys;
  P.k_hs = a->k_stride1 * 2 * heads;
  P.kr_ts = (a->rope_dim > 0 ? a->kr_stride0 : a->k_stride0) * 2 * keys;
  P.v_ts = a->v_stride0 * 2 * keys;
  P.v_hs = a->v_stride1 * 2 * heads;
  P.tokens = (int32_t)a->num_tokens;
  P.keys = (int32_t)a->num_keys;
  P.seqs = (int32_t)a->num_seqs;
  P.heads = (int32_t)a->num_heads;
  P.dim = (int32_t)a->key_dim;
  P.rope = (int32_t)a->rope_dim;
  P.vdim = (int32_t)a->value_dim;
  const int waves = waves_of(a->num_tokens, a->num_keys, a->num_seqs, a->num_heads);
  P.programs = (int32_t)programs_of(a->num_tokens, a->num_keys, a->num_seqs, a->num_heads);
  int64_t reach = 64;
  while (reach < a->num_seqs) reach *= 64;
  P.search_top = (int32_t)(reach / 64);
  P.scale = (float)(std::fabs(a->scale) * 1.4426950408889634074);
  P.vanish = P.scale == 0.0f;
  if (P.vanish) P.scale = 1.0f;
  P.flip = a->scale < 0 ? 0x80008000u : 0u;
  P.causal = a->causal != 0;
  P.splits = splits_of(a->num_tokens, a->num_keys, a->num_seqs, a->num_heads);
  P.partial = static_cast<float*>(workspace);
  const bool wide = std::max(a->key_dim, a->value_dim) > 64, rope = a->rope_dim > 32;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a->dtype == KDACONV_BF16)
    launch<KDACONV_BF16>(P, wide, rope, waves, st);
  else
    launch<KDACONV_F16>(P, wide, rope, waves, st);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}
