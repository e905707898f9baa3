// Absorbed latent attention: checks of arguments and the C entry points. include/kdaconv.h
// states the operator.
#include "latent_attention.h"

#include <algorithm>

namespace kdaconv {
namespace {

constexpr int64_t kSharedBytes = kWorkers * 2 * sizeof(Shared);

bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Blocks of 16 rows per workgroup: as many as a sequence fills on average, up to 4. Every block
// reads the sequence's keys once; 8 blocks' sums and queries are more than the registers hold. The
// average serves unlike sequences too (12 heads, 4096 keys each): 255 decode rows take 226 us, a chunk
// of 512 tokens 103, both in one call 319, though its decode rows are in blocks of 64.
int blocks_of(int64_t tokens, int64_t seqs, int64_t heads) {
  const int64_t rows = tokens * heads;
  return rows <= 16 * seqs ? 1 : rows <= 32 * seqs ? 2 : 4;
}

int validate_attend(const kdaconv_latent_args* a, bool update) {
  if (a == nullptr) return KDACONV_EINVAL;
  if (a->num_tokens < 0 || a->num_seqs < 0 || a->num_heads < 0 || a->pages_per_seq < 0) return KDACONV_EINVAL;
  if (update && a->num_tokens != a->num_seqs) return KDACONV_EINVAL;
  if (a->scale != a->scale) return KDACONV_EINVAL;
  const bool nothing = a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0;
  const int rc = validate_cache(&a->cache, !nothing);
  if (rc != KDACONV_OK) return rc;
  const struct {
    int64_t count, stride;
  } axes[] = {{a->num_tokens, a->ql_stride0}, {a->num_tokens, a->qr_stride0}, {a->num_heads, a->ql_stride1},
              {a->num_heads, a->qr_stride1}, {a->num_seqs, a->table_stride}};
  for (const auto& axis : axes)
    if (axis.count > 1 && axis.stride < 0) return KDACONV_EUNSUPPORTED;
  if (a->num_seqs > INT32_MAX / 2 || a->pages_per_seq > INT32_MAX) return KDACONV_EUNSUPPORTED;
  // Rows are counted in 31 bits.
  if (a->num_tokens > INT32_MAX / 4 || a->num_heads > 65535 || a->num_tokens * a->num_heads > INT32_MAX / 4)
    return KDACONV_EUNSUPPORTED;
  if (nothing) return KDACONV_OK;
  if (!a->q_latent || (a->cache.rope_dim > 0 && !a->q_rope) || !a->seq_lens || !a->out ||
      (a->pages_per_seq > 0 && !a->block_table) || (!update && !a->query_start_loc))
    return KDACONV_EINVAL;
  if (!aligned_to(a->q_latent, 2) || (a->cache.rope_dim > 0 && !aligned_to(a->q_rope, 2)) || !aligned_to(a->out, 2) ||
      !aligned_to(a->seq_lens, 4) || !aligned_to(a->block_table, 4) || (!update && !aligned_to(a->query_start_loc, 4)))
    return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

template <int kF, int kLatent, int kQ>
void launch(const AttendParams& P, bool e4m3, hipStream_t st) {
  if (e4m3)
    launch_attend<kF, kLatent, kQ, true>(P, st);
  else
    launch_attend<kF, kLatent, kQ, false>(P, st);
}

template <int kF, int kLatent>
void launch(const AttendParams& P, int blocks, bool e4m3, hipStream_t st) {
  if (blocks == 1)
    launch<kF, kLatent, 1>(P, e4m3, st);
  else if (blocks == 2)
    launch<kF, kLatent, 2>(P, e4m3, st);
  else
    launch<kF, kLatent, 4>(P, e4m3, st);
}

// Two sizes of kernel: registers and LDS of 512 channels serve all above 256, whose products are the
// channels' that are not there too. 37 decode steps over 90001 keys, 12 heads: 256 channels 30 us,
// 384 35, 512 37.
template <int kF>
void launch(const AttendParams& P, int latent, int blocks, bool e4m3, hipStream_t st) {
  if (latent <= 256)
    launch<kF, 256>(P, blocks, e4m3, st);
  else
    launch<kF, 512>(P, blocks, e4m3, st);
}

int attend(const kdaconv_latent_args* a, bool update, void* workspace, int64_t workspace_bytes, hipStream_t st) {
  const int rc = kdaconv_latent_attention_validate(a, update, workspace, workspace_bytes);
  if (rc != KDACONV_OK || a->num_tokens == 0 || a->num_seqs == 0 || a->num_heads == 0) return rc;
  AttendParams P;
  P.C = cache_view(&a->cache);
  P.T = PageTable{a->block_table, a->table_stride * (a->num_seqs > 1), (int32_t)a->pages_per_seq};
  P.ql = static_cast<const char*>(a->q_latent);
  P.qr = static_cast<const char*>(a->q_rope);
  P.out = static_cast<char*>(a->out);
  P.seq_lens = a->seq_lens;
  P.qsl = update ? nullptr : a->query_start_loc;
  P.shared = static_cast<Shared*>(workspace);
  P.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSharedBytes);
  const int64_t tokens = a->num_tokens > 1, heads = a->num_heads > 1;
  P.ql_ts = a->ql_stride0 * 2 * tokens;
  P.ql_hs = a->ql_stride1 * 2 * heads;
  P.qr_ts = a->qr_stride0 * 2 * tokens;
  P.qr_hs = a->qr_stride1 * 2 * heads;
  P.tokens = (int32_t)a->num_tokens;
  P.seqs = (int32_t)a->num_seqs;
  P.workers = kWorkers;
  P.most_keys = (int32_t)std::min<int64_t>(kMostKeys, a->pages_per_seq * a->cache.page_size);
  P.heads = divider_of((uint32_t)a->num_heads);
  P.scale = (float)(a->scale * 1.4426950408889634074);
  const int blocks = blocks_of(a->num_tokens, a->num_seqs, a->num_heads);
  // What all sequences together can have at most: rows fill at most that many blocks.
  const int64_t most_blocks = a->num_tokens * a->num_heads / (16 * blocks) + std::min(a->num_tokens, a->num_seqs);
  P.shift = 0;
  while (most_blocks * ((P.most_keys >> P.shift) / step_keys(blocks) + 1 + kBlockUnits) > INT32_MAX) ++P.shift;
  if (a->cache.dtype == KDACONV_BF16)
    launch<KDACONV_BF16>(P, (int)a->cache.latent_dim, blocks, a->cache.e4m3 != 0, st);
  else
    launch<KDACONV_F16>(P, (int)a->cache.latent_dim, blocks, a->cache.e4m3 != 0, st);
  return hipGetLastError() == hipSuccess ? KDACONV_OK : KDACONV_ELAUNCH;
}

}  // namespace
}  // namespace kdaconv

using namespace kdaconv;

extern "C" int64_t kdaconv_latent_attention_workspace(int64_t num_tokens, int64_t num_seqs, int64_t num_heads,
                                                      int64_t latent_dim) {
  if (num_tokens <= 0 || num_seqs <= 0 || num_heads <= 0 || latent_dim <= 0) return 0;
  const Partial part{16 * blocks_of(num_tokens, num_seqs, num_heads), (int)latent_dim};
  return kSharedBytes + 2 * kWorkers * part.floats() * (int64_t)sizeof(float);
}

extern "C" int kdaconv_latent_attention_validate(const kdaconv_latent_args* args, int update, const void* workspace,
                                                 int64_t workspace_bytes) {
  const int rc = validate_attend(args, update != 0);
  if (rc != KDACONV_OK) return rc;
  const int64_t need = kdaconv_latent_attention_workspace(args->num_tokens, args->num_seqs, args->num_heads,
                                                          args->cache.latent_dim);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KDACONV_EINVAL;
  if (need > 0 && !aligned_to(workspace, 256)) return KDACONV_EUNSUPPORTED;
  return KDACONV_OK;
}

extern "C" int kdaconv_latent_attention(const kdaconv_latent_args* args, void* workspace, int64_t workspace_bytes,
                                        kdaconv_stream_t stream) {
  return attend(args, false, workspace, workspace_bytes, reinterpret_cast<hipStream_t>(stream));
}

extern "C" int kdaconv_latent_attention_update(const kdaconv_latent_args* args, void* workspace,
                                               int64_t workspace_bytes, kdaconv_stream_t stream) {
  return attend(args, true, workspace, workspace_bytes, reinterpret_cast<hipStream_t>(stream));
}
