/*
 * libkdaconv: the packed varlen causal depthwise width-4 convolution of the
 * KDA prefill (the short convolution over the packed Q|K|V columns of the
 * in_proj output), for AMD Instinct MI355X (gfx950).
 *
 * Operation (page "vllm.models.kimi_k3.nvidia.ops.kda_conv": module docstring,
 * the packed_causal_conv1d_fn docstring and source, and
 * packed_causal_conv1d_supported for the admitted dtypes):
 *   For every sequence s, owning rows [qsl[s], qsl[s+1]) of x, and every channel c
 *   of dim = parts * part_dim channels, with e = (3 history values) ++ (the
 *   sequence's inputs widened to FP32):
 *     acc  = bias[c] (or +0.0f); then acc = fma(w[c][k], e[t-3+k], acc) for k = 0..3
 *     y    = SiLU(acc) = acc / (1 + exp(-acc)), each step in binary32 (or y = acc)
 *     out[c / part_dim][t][c % part_dim] = y in x's format: rounded to bf16 or
 *            fp16 to nearest even (fp16 keeps subnormals and overflows to
 *            infinity), or y itself for FP32
 *   The history is conv_states[cache_indices[s]][c][0..2] (index 0 oldest) when
 *   has_initial_state[s] is set, zeros otherwise. After the call that line holds
 *   the last three values of e. A sequence whose line equals null_block_id (when
 *   has_null_block is set) runs from zeros and leaves the states alone. A
 *   zero-length sequence does nothing. The result is bit-identical to a plain
 *   FP32 evaluation of these steps with a correctly rounded exp. NaN results are
 *   stored as the format's canonical quiet NaN (0x7FC0, 0x7E00, 0x7FC00000).
 *   bf16 and FP32 inputs widen bit for bit; fp16 inputs widen by the IEEE 754
 *   conversion (exact for numbers, a signalling NaN becomes quiet). The state
 *   receives the widened values.
 *
 * Conventions for every entry point:
 *   - Sizes and strides count ELEMENTS, not bytes. Pointers are DEVICE pointers
 *     unless stated otherwise, owned by the caller; the library allocates no
 *     memory, keeps no state between calls, never synchronises and never reads
 *     device data on the host. Work is queued on `stream` (NULL = the default
 *     stream) and the call returns before it finishes.
 *   - The launch geometry depends only on num_tokens, num_seqs and dim, so a
 *     call can be captured in a HIP graph and replayed with new device data of
 *     the same shapes.
 *   - Return values are the kdaconv_status codes below. Nothing is launched when
 *     a check fails; the output and the states are then left as they were.
 *   - Thread-safe: calls on different streams may run concurrently as long as
 *     they do not write the same memory.
 */
#ifndef KDACONV_H_
#define KDACONV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as hipStream_t. */
struct ihipStream_t;
typedef struct ihipStream_t* kdaconv_stream_t;

typedef enum kdaconv_status {
  KDACONV_OK = 0,
  KDACONV_EINVAL = 1,       /* an argument is outside its documented range */
  KDACONV_EUNSUPPORTED = 2, /* meaningful, but a layout or size this library does not handle */
  KDACONV_ELAUNCH = 3       /* the HIP runtime refused the launch */
} kdaconv_status;

typedef enum kdaconv_activation {
  KDACONV_ACT_NONE = 0,
  KDACONV_ACT_SILU = 1
} kdaconv_activation;

/* Element format of x and of the output (the output takes x's format). */
typedef enum kdaconv_dtype {
  KDACONV_BF16 = 0,
  KDACONV_F16 = 1,
  KDACONV_F32 = 2
} kdaconv_dtype;

/*
 * The convolution (packed_causal_conv1d_fn on the page named above).
 *
 * x                  elements of format dtype; element (t, c) at
 *                    x[t * x_row_stride + c], rows t < num_tokens, channels c < dim.
 *                    Only columns [0, dim) are read. x_row_stride >= dim, any
 *                    value (page: unit column stride, any row stride). x must be
 *                    aligned to its element size (else EUNSUPPORTED). 4 channels
 *                    move as one vector whatever the alignment, so a Q|K|V slice
 *                    may start at any column; vectors at addresses that are not
 *                    multiples of 8 bytes (bf16, fp16) or 16 bytes (FP32) cost
 *                    some speed.
 * dtype              KDACONV_BF16, KDACONV_F16 or KDACONV_F32 (else EINVAL): the
 *                    format of x and of out.
 * weight             FP32; tap k of channel c at weight[c * weight_stride0 +
 *                    k * weight_stride1] (page layout [channel, width], width 4).
 * bias               FP32 (dim,) contiguous, or NULL for none.
 * conv_states        FP32, logical shape (num_cache_lines, dim, 3): history k of
 *                    channel c of line l at conv_states[l * cs_stride0 +
 *                    c * cs_stride1 + k * cs_stride2]. Read and written in place.
 *                    Any layout the strides describe: (lines, dim, 3) contiguous and
 *                    "dim first" (lines, 3, dim) take vector paths; a state wider
 *                    than 3 (lines, dim, W) passes its strides, entries 0..2 are the
 *                    history and the rest are not touched (the page's launch passes
 *                    the three strides and not the width).
 * query_start_loc    int32 (num_seqs + 1): sequence s owns rows [qsl[s], qsl[s+1]).
 *                    Must be non-decreasing with qsl[num_seqs] <= num_tokens; rows
 *                    outside every sequence are neither read nor written.
 * cache_indices      int32, the line of sequence s at cache_indices[s *
 *                    cache_indices_stride]. Live lines (not the null block) must be
 *                    distinct within a call. A line outside [0, num_cache_lines) is
 *                    treated like the null block (no state read or write).
 * has_initial_state  one byte per sequence (nonzero = start from the stored line),
 *                    or NULL: every sequence starts from zeros.
 * part_dim           channels per output plane; dim % part_dim == 0 (else EINVAL)
 *                    and part_dim % 8 == 0 (else EUNSUPPORTED).
 * activation         KDACONV_ACT_NONE or KDACONV_ACT_SILU (else EINVAL).
 * has_null_block,
 * null_block_id      when has_null_block != 0, sequences whose line equals
 *                    null_block_id skip the state (page: HAS_NULL_BLOCK).
 * out                elements of format dtype, dense (dim / part_dim, num_tokens,
 *                    part_dim), aligned to the element size (see x). Rows no
 *                    sequence owns are left unwritten.
 *
 * Device-data preconditions (not checked; violating them gives unspecified
 * values but no access outside the buffers described above): query_start_loc
 * non-decreasing and within [0, num_tokens]; distinct live lines.
 * num_tokens == 0, num_seqs == 0 or dim == 0 returns KDACONV_OK with no launch.
 */
int kdaconv_packed_causal_conv1d(
    const void* x, int dtype, int64_t num_tokens, int64_t dim, int64_t x_row_stride,
    const float* weight, int64_t weight_stride0, int64_t weight_stride1,
    const float* bias,
    float* conv_states, int64_t num_cache_lines,
    int64_t cs_stride0, int64_t cs_stride1, int64_t cs_stride2,
    const int32_t* query_start_loc, int64_t num_seqs,
    const int32_t* cache_indices, int64_t cache_indices_stride,
    const uint8_t* has_initial_state,
    int64_t part_dim, int activation, int has_null_block, int64_t null_block_id,
    void* out, kdaconv_stream_t stream);

/*
 * The decode step: the packed causal conv1d update of one token per sequence
 * (page "vllm.models.kimi_k3.amd.ops.kda_decode": the first of the three steps its
 * fused decode kernel replaces), with the FP32 state of the prefill op. Sequence b
 * of the batch owns row b of x. Its result is that of kdaconv_packed_causal_conv1d
 * on the same x with query_start_loc = {0, 1, ..., batch} and every
 * has_initial_state set: the history is the stored line (zeros for the null block,
 * whose line is neither read nor written), out[c / part_dim][b][c % part_dim] is the
 * activated, rounded tap sum, and the line becomes entries 1, 2 and the new token.
 * With an FP32 state the arithmetic is FP32 for every x dtype (page
 * "vllm.models.kimi_k3.nvidia.ops.kda_conv", packed_causal_conv1d_supported's note).
 * The bf16 state of the decode page's kernel is taken by
 * kdaconv_packed_causal_conv1d_update_bf16_state below.
 *
 * x                  elements of format dtype, (batch, dim) at row stride
 *                    x_row_stride (alignment as for the prefill op).
 * weight, bias,
 * conv_states,
 * cache_indices,
 * part_dim,
 * activation,
 * has_null_block,
 * null_block_id      as for kdaconv_packed_causal_conv1d; cache_indices has one
 *                    entry per sequence of the batch.
 * out                elements of format dtype, dense (dim / part_dim, batch, part_dim),
 *                    aligned to the element size.
 *
 * Precondition (not checked): live lines distinct within the batch.
 * batch == 0 or dim == 0 returns KDACONV_OK with no launch. Status codes and
 * their checks are those of kdaconv_packed_causal_conv1d, with batch in place of
 * num_tokens and num_seqs.
 */
int kdaconv_packed_causal_conv1d_update(
    const void* x, int dtype, int64_t batch, int64_t dim, int64_t x_row_stride,
    const float* weight, int64_t weight_stride0, int64_t weight_stride1,
    const float* bias,
    float* conv_states, int64_t num_cache_lines,
    int64_t cs_stride0, int64_t cs_stride1, int64_t cs_stride2,
    const int32_t* cache_indices, int64_t cache_indices_stride,
    int64_t part_dim, int activation, int has_null_block, int64_t null_block_id,
    void* out, kdaconv_stream_t stream);

/*
 * The decode step with the operands of the fused decode kernel on page
 * "vllm.models.kimi_k3.amd.ops.kda_decode": a bf16 conv state and the FP32 weight
 * mirrored width-major (is_fused_kda_decode_supported admits a bf16 input with a bf16
 * conv state, not dim-first; make_decode_conv1d_weight_loader's docstring gives the
 * weight as [qkv, width, channel]). The page prints no arithmetic. The reading taken:
 * the state's bf16 values and the token widen exactly to FP32 and go through the same
 * FP32 chain, activation and rounding as kdaconv_packed_causal_conv1d_update, so the
 * output equals that call on the widened state; the line then holds entries 1 and 2
 * and the token, whose words are kept unchanged (they are bf16 values already; a NaN
 * keeps its payload).
 *
 * x                  bf16 (batch, dim) at row stride x_row_stride (alignment as for
 *                    the prefill op). dtype must be KDACONV_BF16 (the page's gate);
 *                    fp16 and FP32 give EUNSUPPORTED, unknown codes EINVAL.
 * weight             FP32; tap k of channel c at weight[(c / part_dim) *
 *                    weight_part_stride + (c % part_dim) * weight_stride0 + k *
 *                    weight_stride1]. The page's width-major (dim / part_dim, 4,
 *                    part_dim) array is part stride 4 * part_dim, stride0 1, stride1
 *                    part_dim, and the prefill op's (dim, 4) array is 4 * part_dim,
 *                    4, 1; both take vector paths when 16-byte aligned, any other
 *                    strides a scalar one.
 * conv_states        bf16 words, logical shape (num_cache_lines, dim, 3): history k
 *                    of channel c of line l at conv_states[l * cs_stride0 + c *
 *                    cs_stride1 + k * cs_stride2]; (lines, dim, 3) contiguous and
 *                    8-byte aligned takes a vector path, any other strides a scalar
 *                    one. Read and written in place.
 * bias, cache_indices,
 * part_dim, activation,
 * has_null_block,
 * null_block_id, out as for kdaconv_packed_causal_conv1d_update (out is bf16).
 *
 * Precondition (not checked): live lines distinct within the batch.
 * batch == 0 or dim == 0 returns KDACONV_OK with no launch. Status codes and their
 * checks are those of kdaconv_packed_causal_conv1d_update, and a negative
 * weight_part_stride gives EUNSUPPORTED.
 */
int kdaconv_packed_causal_conv1d_update_bf16_state(
    const void* x, int dtype, int64_t batch, int64_t dim, int64_t x_row_stride,
    const float* weight, int64_t weight_part_stride, int64_t weight_stride0,
    int64_t weight_stride1, const float* bias,
    uint16_t* conv_states, int64_t num_cache_lines,
    int64_t cs_stride0, int64_t cs_stride1, int64_t cs_stride2,
    const int32_t* cache_indices, int64_t cache_indices_stride,
    int64_t part_dim, int activation, int has_null_block, int64_t null_block_id,
    void* out, kdaconv_stream_t stream);

/*
 * Host-only check of the same arguments (page: packed_causal_conv1d_supported):
 * returns the status kdaconv_packed_causal_conv1d would return before launching.
 * Pointers are only compared with NULL and tested for alignment, never
 * dereferenced, so host addresses may stand in for device ones. Makes no HIP call.
 */
int kdaconv_validate(
    const void* x, int dtype, int64_t num_tokens, int64_t dim, int64_t x_row_stride,
    const float* weight, int64_t weight_stride0, int64_t weight_stride1,
    const float* bias,
    const float* conv_states, int64_t num_cache_lines,
    int64_t cs_stride0, int64_t cs_stride1, int64_t cs_stride2,
    const int32_t* query_start_loc, int64_t num_seqs,
    const int32_t* cache_indices, int64_t cache_indices_stride,
    const uint8_t* has_initial_state,
    int64_t part_dim, int activation, int has_null_block, int64_t null_block_id,
    const void* out);

/*
 * The device map from an FP32 accumulator to the stored word of format dtype,
 * exactly as the convolution kernel applies it (SiLU or none, then the format's
 * rounding; module docstring of the page named above), evaluated for the `count`
 * FP32 bit patterns first, first + 1, ... (wrapping at 2^32). out: device array of
 * `count` words (uint16 for bf16 and fp16, uint32 for FP32), 16-byte aligned.
 * count must be a multiple of 8 (else EINVAL). Used to check the kernel's
 * activation against a reference on every input.
 */
int kdaconv_activation_map(uint32_t first, int64_t count, int activation, int dtype, void* out,
                           kdaconv_stream_t stream);

/*
 * The gated delta rule: the operator of a KDA layer that reads the convolution's planes.
 * Per value head h, with a state S of head_dim rows (key channels) by head_dim columns
 * (value channels), for every token t of a sequence:
 *     a_t = exp(log decay)             per key channel, from g:
 *           KDACONV_GATE_LOG           log decay = g
 *           KDACONV_GATE_SOFTPLUS      log decay = -exp(a_log[h]) * softplus(g + dt_bias[h])
 *           KDACONV_GATE_BOUNDED       log decay = lower_bound *
 *                                          sigmoid(exp(a_log[h]) * (g + dt_bias[h]))
 *     k_t, q_t = k and q of head h / (num_heads / num_qk_heads), each divided by
 *           sqrt(|.|^2 + l2_eps) when l2_eps >= 0
 *     b_t = beta, or sigmoid(beta) with beta_logits
 *     S'  = diag(a_t) S;   u_t = b_t (v_t - S'^T k_t);   S = S' + k_t u_t^T
 *     out_t = scale * S^T q_t          rounded to the format of q, k and v
 * Sequences, lines, initial states and the null block are those of
 * kdaconv_packed_causal_conv1d: sequence s owns rows [qsl[s], qsl[s+1]), starts from
 * states[cache_indices[s]] when has_initial_state[s] is set (else zeros) and leaves its
 * last S there; a sequence on the null block, or on a line outside the state array, runs
 * from zeros and leaves the states alone. A sequence without tokens leaves what it starts
 * from: its line as it is, or zeros there without an initial state. States, sums and norms
 * are held in FP32 or more; matrix products take FP32 values as pairs of FP16 values (22
 * bits) and sum in FP32; only out is rounded to its format. Errors of the prefill are about
 * 2^-22 of the largest value that a column of the state, or of v, has within 32 tokens. Keys and
 * queries taken as they are (l2_eps < 0) lose bits below a length of 2^-118.
 * A value that is not finite reaches what the steps above take it to, tokens from its own on,
 * and no token before it nor another sequence.
 * A log decay below -104 acts as -104 (its exp is zero in FP32, as is -infinity's). Log
 * decays given as they are (KDACONV_GATE_LOG) are at most 0; positive ones are not looked for
 * and may leave the range of the prefill's FP16 pairs.
 *
 * All strides count elements. Those of q, k, v, g and beta are 0 to 2^23 - 1 (else
 * EUNSUPPORTED); of an axis of one entry they are not looked at.
 */
typedef enum kdaconv_gate {
  KDACONV_GATE_LOG = 0,
  KDACONV_GATE_SOFTPLUS = 1,
  KDACONV_GATE_BOUNDED = 2
} kdaconv_gate;

typedef struct kdaconv_rule_args {
  const void* q;    /* (num_tokens, num_qk_heads, head_dim), last axis contiguous */
  const void* k;    /* as q */
  const void* v;    /* (num_tokens, num_heads, head_dim), last axis contiguous */
  const void* g;    /* (num_tokens, num_heads, head_dim); g_stride2 is 1, or 0 for one
                       gate per head */
  const void* beta; /* (num_tokens, num_heads) */
  const float* a_log;   /* (num_heads), contiguous; NULL with KDACONV_GATE_LOG */
  const float* dt_bias; /* (num_heads, head_dim), contiguous, or NULL for none */
  float* states;        /* (num_cache_lines, num_heads, head_dim, head_dim) [key][value];
                           the last two axes are contiguous */
  const int32_t* query_start_loc;   /* (num_seqs + 1); ignored by the update */
  const int32_t* cache_indices;     /* (num_seqs) */
  const uint8_t* has_initial_state; /* (num_seqs) or NULL (none); the update takes every
                                       sequence from its stored line */
  void* out;            /* (num_tokens, num_heads, head_dim), contiguous */
  int64_t num_tokens, num_seqs, num_heads, num_qk_heads, head_dim;
  int64_t q_stride0, q_stride1, k_stride0, k_stride1, v_stride0, v_stride1;
  int64_t g_stride0, g_stride1, g_stride2, beta_stride0, beta_stride1;
  int64_t num_cache_lines, state_stride0, state_stride1;
  int64_t cache_indices_stride;
  int64_t null_block_id;
  double scale, l2_eps, lower_bound;
  int32_t dtype;      /* kdaconv_dtype of q, k, v and out */
  int32_t gate_dtype; /* of g: dtype, or KDACONV_F32 */
  int32_t beta_dtype; /* of beta: dtype, or KDACONV_F32 */
  int32_t gate;       /* kdaconv_gate */
  int32_t beta_logits;
  int32_t has_null_block;
} kdaconv_rule_args;

/*
 * Bytes of device scratch memory that kdaconv_gated_delta_rule needs for these sizes (0
 * for none; about 60 KB per 32 tokens and head of 128, 35 KB per head of 64). It grows with the
 * call: 0.4 GB for 16384 tokens of 12 heads of 128, 16 GB for 131072 of 64. The scratch holds no
 * state between calls; calls that may run at the same time need scratch memories of their own.
 * Aligned to 256 bytes.
 */
int64_t kdaconv_gated_delta_rule_workspace(int64_t num_tokens, int64_t num_seqs,
                                           int64_t num_heads, int64_t head_dim);

/*
 * The rule over packed sequences (prefill). head_dim is 64 or 128 and num_heads a
 * multiple of num_qk_heads (else EUNSUPPORTED and EINVAL). Sizes come from the host
 * arguments alone, so a call can be captured in a graph. Preconditions on device data as
 * for kdaconv_packed_causal_conv1d. num_tokens, num_seqs or num_heads of 0: KDACONV_OK
 * with no launch (a call without any token leaves all states alone). out may not overlap an
 * input. From (num_tokens / 32 + num_seqs) * num_heads = 2^23 on a call may be refused
 * (EUNSUPPORTED).
 */
int kdaconv_gated_delta_rule(const kdaconv_rule_args* args, void* workspace,
                             int64_t workspace_bytes, kdaconv_stream_t stream);

/*
 * The rule for one token per sequence (decode): row s of q, k, v, g, beta and out belongs
 * to sequence s, num_seqs equals num_tokens (else EINVAL), and every sequence continues
 * from its stored line (zeros for the null block). query_start_loc and has_initial_state
 * are not read. No scratch memory. Sequences times heads below 2^23 (else EUNSUPPORTED).
 */
int kdaconv_gated_delta_rule_update(const kdaconv_rule_args* args, kdaconv_stream_t stream);

/* The status either call would return before launching (update != 0: the update's). No
 * HIP call; device pointers are only compared with NULL and tested for alignment. */
int kdaconv_gated_delta_rule_validate(const kdaconv_rule_args* args, int update,
                                      const void* workspace, int64_t workspace_bytes);

typedef enum kdaconv_norm_gate {
  KDACONV_NORM_GATE_NONE = 0,
  KDACONV_NORM_GATE_SIGMOID = 1,
  KDACONV_NORM_GATE_SILU = 2
} kdaconv_norm_gate;

/*
 * The norm after the rule: for every token t and head h,
 *     y = x / sqrt(mean(x^2) + eps) * weight * act(gate)
 * over the head's `dim` channels, computed in FP32 and rounded once to dtype. act is the
 * sigmoid, or gate * sigmoid(gate), or absent (gate NULL with KDACONV_NORM_GATE_NONE).
 *
 * x, gate   format dtype; (t, h, c) at t * stride0 + h * stride1 + c.
 * weight    FP32 (dim) contiguous, or NULL for ones.
 * out       format dtype, (num_tokens, num_heads, dim) contiguous; may be x itself when
 *           x is laid out like it.
 * dim       a positive multiple of 8, at most 512 (else EUNSUPPORTED, as are more than
 *           2^28 - 16 tokens times heads).
 */
int kdaconv_gated_rms_norm(const void* x, int dtype, int64_t num_tokens, int64_t num_heads,
                           int64_t dim, int64_t x_stride0, int64_t x_stride1, const void* gate,
                           int64_t gate_stride0, int64_t gate_stride1, int activation,
                           const float* weight, double eps, void* out, kdaconv_stream_t stream);

/*
 * The residual addition and the norm before a block: for every row t,
 *     h = residual + residual_scale * x;   y = h / sqrt(mean(h^2) + eps) * weight
 * with h in FP32; residual is replaced by h rounded to dtype, and out by y rounded once
 * (y comes from the FP32 h). residual may be NULL: h = residual_scale * x, kept nowhere.
 *
 * x, residual  format dtype; row t at t * stride, columns contiguous.
 * weight       FP32 (hidden) contiguous, or NULL for ones.
 * out          format dtype, (num_tokens, hidden) contiguous.
 * hidden       1 to 16384 (else EUNSUPPORTED, as are 2^24 tokens and more).
 */
int kdaconv_residual_rms_norm(const void* x, int dtype, int64_t num_tokens, int64_t hidden,
                              int64_t x_stride, void* residual, int64_t residual_stride,
                              double residual_scale, const float* weight, double eps, void* out,
                              kdaconv_stream_t stream);

/*
 * Latent attention: the attention layer that alternates with KDA layers. All heads' keys and
 * values come from one latent vector of latent_dim channels and one rotated vector of rope_dim
 * channels a token, which are what its cache holds.
 *
 * Rotary positions. Channels [offset, offset + rotary) of every head are turned in pairs, pair
 * i by the angle a_i = positions[t] * inv_freq[i]:
 *     (u, v) -> (scale * (u cos a_i - v sin a_i), scale * (u sin a_i + v cos a_i))
 * Pair i is channels (2 i, 2 i + 1) with `interleaved`, else (i, i + rotary / 2), counted from
 * offset. The angle is taken in FP64 and reduced to a turn there, so far positions keep their
 * precision; products are FP32, rounded once. The other channels are copied (left alone where
 * out is x itself, laid out alike).
 *
 * x, out     (num_tokens, num_heads, head_dim), element (t, h, c) at t * stride0 +
 *            h * stride1 + c; format dtype (bf16, fp16 or FP32). out may be x with x's strides;
 *            it may not overlap x otherwise, nor itself.
 * positions  (num_tokens) int32, or int64 with positions_64; any value. Angles are off by 2^-26 of a
 *            turn at most up to 2^53 (beyond, positions round to FP64).
 * inv_freq   (rotary / 2) FP32. rotary is even, 2 to 512 (else EINVAL, EUNSUPPORTED), and
 *            offset + rotary <= head_dim (else EINVAL). num_heads is below 2^16, head_dim at most
 *            2^16 and their product below 2^31 - 256 (else EUNSUPPORTED).
 */
int kdaconv_rotary_embedding(const void* x, int dtype, int64_t num_tokens, int64_t num_heads,
                             int64_t head_dim, int64_t x_stride0, int64_t x_stride1,
                             const void* positions, int positions_64, const float* inv_freq,
                             int64_t rotary, int64_t offset, int interleaved, double scale,
                             void* out, int64_t out_stride0, int64_t out_stride1,
                             kdaconv_stream_t stream);

/*
 * A paged cache. Slot s of it is place s % page_size of page s / page_size. With e4m3 a latent
 * is held in 8 bits (OCP E4M3) and a scale byte b for each 32 channels stands for 2^(b - 127);
 * 255 is no scale. rope_dim may be 0. Strides count elements of the tensor they belong to.
 *
 * latent_dim is a multiple of 8 (32 with e4m3), 8 to 512, and rope_dim one of 8, 0 to 64 (else
 * EUNSUPPORTED). Latents and rotated parts lie at multiples of 16 bytes, page for page and slot
 * for slot (else EUNSUPPORTED). num_pages * page_size is below 2^31 (else EUNSUPPORTED).
 */
typedef struct kdaconv_latent_cache {
  void* latents;   /* (num_pages, page_size, latent_dim): dtype, or e4m3 codes */
  void* ropes;     /* (num_pages, page_size, rope_dim): dtype */
  uint8_t* scales; /* (num_pages, page_size, latent_dim / 32) with e4m3, else ignored */
  int64_t num_pages, page_size, latent_dim, rope_dim;
  int64_t latents_stride0, latents_stride1, ropes_stride0, ropes_stride1;
  int64_t scales_stride0, scales_stride1;
  int32_t dtype; /* KDACONV_BF16 or KDACONV_F16 */
  int32_t e4m3;
} kdaconv_latent_cache;

/*
 * Writes tokens into the cache. Of token t the latent
 *     y = latent / sqrt(mean(latent^2) + eps) * weight      (y = latent with eps < 0)
 * and the rotated part (kdaconv_rotary_embedding with one head of rope_dim channels; as it is
 * without inv_freq) go to slot slots[t]; a slot outside the cache is left out. The norm is
 * worked out in FP64 and y is its FP32 rounding, so that codes do not depend on the order of a
 * sum. y is rounded to dtype, or with e4m3 each block of 32 is held as codes of y / 2^e, rounded
 * to nearest even, where e is the smallest integer >= -100 with max |y| <= 448 * 2^e over the
 * block's finite values (infinities and NaN become the code NaN).
 *
 * latent, rope  (num_tokens, latent_dim) and (num_tokens, rope_dim) of the cache's dtype,
 *               columns contiguous.
 * slots         (num_tokens) int32, or int64 with slots_64; slots in the cache are distinct.
 * weight        FP32 (latent_dim), or NULL for ones.
 */
int kdaconv_latent_cache_write(const kdaconv_latent_cache* cache, const void* latent,
                               int64_t latent_stride, const void* rope, int64_t rope_stride,
                               int64_t num_tokens, const void* slots, int slots_64,
                               const float* weight, double eps, const void* positions,
                               int positions_64, const float* inv_freq, int interleaved,
                               double rope_scale, kdaconv_stream_t stream);

/*
 * Reads sequences back out of the cache: row kv_start_loc[s] + i of out (num_tokens,
 * latent_dim + rope_dim), contiguous, of the cache's dtype, gets token i of sequence s, which
 * lies in slot block_table[s][i / page_size] * page_size + i % page_size. e4m3 values times
 * their scale are rounded once. Rows of sequences past num_tokens, and those no sequence owns,
 * are not written; a token whose page is outside the cache, or past the table's pages_per_seq
 * columns, reads as zeros. out is aligned to 16 bytes (else EUNSUPPORTED).
 */
int kdaconv_latent_cache_read(const kdaconv_latent_cache* cache, const int32_t* block_table,
                              int64_t table_stride, int64_t pages_per_seq,
                              const int32_t* kv_start_loc, int64_t num_seqs, int64_t num_tokens,
                              void* out, kdaconv_stream_t stream);

/*
 * Attention over the paged cache in the absorbed form: queries are already multiplied by the
 * latents' up-projection, and what comes out is still to be multiplied by the values'. Token i of
 * the n new tokens of sequence s (rows [qsl[s], qsl[s+1])), whose latents are in the cache, sees
 * the sequence's first seq_lens[s] - n + i + 1 tokens: for every head
 *     s_t = scale * (q_latent . latent_t + q_rope . rope_t),   out = sum_t softmax(s)_t latent_t
 * A token whose page is outside the cache, or past the table's pages_per_seq columns, is not
 * there; a row that sees none is zero, and so is one whose scores are all -inf. A latent that is
 * not finite reaches no row that does not see it. Rows no sequence owns are not written. Scores, softmax
 * and sums are FP32; its weights (up to 2^8 before the division by their sum) are rounded to
 * dtype for the second product, out is rounded once. 8-bit values times their scale are rounded
 * to dtype, exactly within its range.
 */
typedef struct kdaconv_latent_args {
  kdaconv_latent_cache cache;
  const void* q_latent; /* (num_tokens, num_heads, latent_dim) of the cache's dtype */
  const void* q_rope;   /* (num_tokens, num_heads, rope_dim); ignored if rope_dim is 0 */
  const int32_t* block_table;     /* (num_seqs, pages_per_seq) */
  const int32_t* seq_lens;        /* (num_seqs), up to 2^30 */
  const int32_t* query_start_loc; /* (num_seqs + 1); ignored by the update */
  void* out;                      /* (num_tokens, num_heads, latent_dim), contiguous */
  int64_t num_tokens, num_seqs, num_heads;
  int64_t ql_stride0, ql_stride1, qr_stride0, qr_stride1;
  int64_t table_stride, pages_per_seq;
  double scale;
} kdaconv_latent_args;

/*
 * Bytes of device scratch memory of a call of these sizes: up to 67 MB, 17 MB where sequences
 * have up to 16 rows (tokens times heads) on average. It holds no state between calls; calls that
 * may run at the same time need scratch memories of their own. Aligned to 256 bytes.
 */
int64_t kdaconv_latent_attention_workspace(int64_t num_tokens, int64_t num_seqs, int64_t num_heads,
                                           int64_t latent_dim);

/*
 * New tokens of any number per sequence. The work is split by the lengths on the device: the
 * launch depends on host sizes alone, and a call can be captured in a graph. num_tokens,
 * num_seqs or num_heads of 0: KDACONV_OK with no launch. num_tokens * num_heads is below 2^29
 * (else EUNSUPPORTED).
 */
int kdaconv_latent_attention(const kdaconv_latent_args* args, void* workspace,
                             int64_t workspace_bytes, kdaconv_stream_t stream);

/* One token per sequence (decode): row s belongs to sequence s, num_seqs equals num_tokens (else
 * EINVAL); query_start_loc is not read. */
int kdaconv_latent_attention_update(const kdaconv_latent_args* args, void* workspace,
                                    int64_t workspace_bytes, kdaconv_stream_t stream);

/* The status either call would return before launching (update != 0: the update's). No HIP
 * call; device pointers are only compared with NULL and tested for alignment. */
int kdaconv_latent_attention_validate(const kdaconv_latent_args* args, int update,
                                      const void* workspace, int64_t workspace_bytes);

/*
 * Attention of packed sequences in the expanded form: every head has keys and values of its own
 * (a latent's up-projection), beside the rotated part of the keys that all heads share. Row i of
 * the n queries of sequence s, rows [qsl[s], qsl[s+1]), sees the first m - n + i + 1 of its m
 * keys, rows [ksl[s], ksl[s+1]) of k, k_rope and v, or all of them without `causal`:
 *     s_t = scale * (q[:key_dim] . k_t + q[key_dim:] . k_rope_t),   out = sum_t softmax(s)_t v_t
 * A row that sees none is zero, and so is one whose scores are all -inf; rows no sequence owns are
 * not written. Scores, softmax and sums are FP32; its weights (up to 2^8 before the division by their sum) are rounded to dtype for the
 * second product, out is rounded once. A key or value that is not finite reaches no row that does
 * not see it; a channel of the rows that see such a value is NaN or infinite.
 *
 * key_dim and value_dim are multiples of 8 up to 128, rope_dim is one of 8, 0 to 64 (else
 * EUNSUPPORTED); up to 64, 64 and 32 a smaller kernel serves. k, v and k_rope lie at multiples of
 * 16 bytes, token for token and head for head (else EUNSUPPORTED). Strides count elements and are
 * not negative, those of the tokens of k, k_rope and v below 2^23 (else EUNSUPPORTED); of an axis
 * of one entry they are not looked at.
 */
typedef struct kdaconv_expanded_args {
  const void* q;      /* (num_tokens, num_heads, key_dim + rope_dim), last axis contiguous */
  const void* k;      /* (num_keys, num_heads, key_dim), last axis contiguous */
  const void* k_rope; /* (num_keys, rope_dim), columns contiguous; ignored if rope_dim is 0 */
  const void* v;      /* (num_keys, num_heads, value_dim), last axis contiguous */
  const int32_t* query_start_loc; /* (num_seqs + 1) */
  const int32_t* kv_start_loc;    /* (num_seqs + 1) */
  void* out;          /* (num_tokens, num_heads, value_dim), contiguous */
  int64_t num_tokens, num_keys, num_seqs, num_heads, key_dim, rope_dim, value_dim;
  int64_t q_stride0, q_stride1, k_stride0, k_stride1, kr_stride0, v_stride0, v_stride1;
  double scale;
  int32_t dtype; /* KDACONV_BF16 or KDACONV_F16 */
  int32_t causal;
} kdaconv_expanded_args;

/* The launch depends on host sizes alone, so a call can be captured in a graph. num_tokens,
 * num_seqs or num_heads of 0: KDACONV_OK with no launch. (num_tokens / 128 + num_seqs) *
 * num_heads is below 2^23 (else EUNSUPPORTED). workspace is device memory of at least
 * kdaconv_expanded_attention_workspace bytes, none where that is 0 (else EINVAL), aligned to 256
 * bytes (else EUNSUPPORTED); it holds nothing between calls, but no two calls in flight share it. */
int kdaconv_expanded_attention(const kdaconv_expanded_args* args, void* workspace,
                               int64_t workspace_bytes, kdaconv_stream_t stream);

/* Bytes of scratch memory: 0 but for few rows over many keys, whose keys are split. */
int64_t kdaconv_expanded_attention_workspace(int64_t num_tokens, int64_t num_keys, int64_t num_seqs,
                                             int64_t num_heads, int64_t value_dim);

/* The status the call would return before launching. No HIP call; device pointers are only
 * compared with NULL and tested for alignment. */
int kdaconv_expanded_attention_validate(const kdaconv_expanded_args* args, const void* workspace,
                                        int64_t workspace_bytes);

/* Static English text for a status code. Never NULL. */
const char* kdaconv_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int kdaconv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDACONV_H_ */
