"""The gated delta rule over the convolution's planes: prefill and the single-token step."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._host import DTYPE_CODES, NULL_BLOCK_ID, _call, _fresh_like

#: Added to the squared length of a query or key before its root (qk_l2norm).
L2_EPS = 1e-6

_FLAGS = (torch.bool, torch.uint8)


def _heads(q, k, v, g, beta, states):
    """Checks shapes and types; returns the sizes and the dtype codes."""
    if q.dim() != 3 or v.dim() != 3 or k.shape != q.shape:
        raise ValueError("q and k must be (tokens, qk heads, head_dim) and v (tokens, heads, head_dim)")
    tokens, heads, dim = v.shape
    if q.shape[0] != tokens or q.shape[2] != dim:
        raise ValueError("q, k and v must agree in tokens and head_dim")
    qk_heads = q.shape[1]
    if heads and (qk_heads == 0 or heads % qk_heads):
        raise ValueError(f"the heads of v ({heads}) must be a multiple of those of q and k ({qk_heads})")
    dtype = v.dtype
    if dtype not in DTYPE_CODES or q.dtype != dtype or k.dtype != dtype:
        raise ValueError("q, k and v must share one dtype: bfloat16, float16 or float32")
    if g.dtype != dtype and g.dtype != torch.float32 or beta.dtype != dtype and beta.dtype != torch.float32:
        raise ValueError("g and beta must have the dtype of v, or float32")
    if g.shape != v.shape and g.shape != (tokens, heads):
        raise ValueError("g must be (tokens, heads, head_dim), or (tokens, heads) for one gate per head")
    if beta.shape != (tokens, heads):
        raise ValueError("beta must be (tokens, heads)")
    if states.dtype != torch.float32 or states.dim() != 4 or states.shape[1:] != (heads, dim, dim):
        raise ValueError("states must be float32 (cache lines, heads, head_dim, head_dim)")
    return tokens, heads, qk_heads, dim


def _pack(q, k, v, g, beta, states, cache_indices, query_start_loc, has_initial_state, num_seqs,
          sizes, a_log, dt_bias, lower_bound, beta_logits, qk_l2norm, scale, null_block_id, out):
    """kdaconv_rule_args as bytes, after the checks that need the tensors."""
    tokens, heads, qk_heads, dim = sizes
    qs, ks, vs, gs, bs, ss = (q.stride(), k.stride(), v.stride(), g.stride(), beta.stride(),
                              states.stride())
    if dim > 1 and (qs[2] != 1 or ks[2] != 1 or vs[2] != 1):
        raise ValueError("the last axis of q, k and v must be contiguous")
    per_channel = len(gs) == 3 and gs[2] != 0
    if per_channel and gs[2] != 1:
        raise ValueError("the last axis of g must be contiguous (or have stride 0)")
    if ss[3] != 1 or ss[2] != dim:
        raise ValueError("the last two axes of states must be contiguous")
    if a_log is None:
        if dt_bias is not None or lower_bound is not None:
            raise ValueError("dt_bias and lower_bound need a_log (without it g is the log decay itself)")
        gate = _lib.GATE_LOG
    else:
        gate = _lib.GATE_SOFTPLUS if lower_bound is None else _lib.GATE_BOUNDED
        if a_log.dtype != torch.float32 or a_log.shape != (heads,) or not a_log.is_contiguous():
            raise ValueError("a_log must be a contiguous float32 (heads,) tensor")
        if dt_bias is not None and (dt_bias.dtype != torch.float32 or not dt_bias.is_contiguous()
                                    or dt_bias.shape not in ((heads, dim), (heads * dim,))):
            raise ValueError("dt_bias must be a contiguous float32 (heads, head_dim) tensor or None")
        if lower_bound is not None and not lower_bound <= 0:
            raise ValueError("lower_bound must not be positive")
    if (cache_indices.dtype != torch.int32 or cache_indices.dim() != 1
            or cache_indices.shape[0] < num_seqs):
        raise ValueError("cache_indices must be a 1-D int32 tensor with one entry per sequence")
    device = v.get_device()
    if device < 0:
        raise ValueError("v must be a GPU tensor")
    if (q.get_device() != device or k.get_device() != device or g.get_device() != device
            or beta.get_device() != device or states.get_device() != device
            or cache_indices.get_device() != device
            or query_start_loc is not None and query_start_loc.get_device() != device
            or has_initial_state is not None and has_initial_state.get_device() != device
            or a_log is not None and a_log.get_device() != device
            or dt_bias is not None and dt_bias.get_device() != device):
        raise ValueError("all tensors must be on the device of v")
    code = DTYPE_CODES[v.dtype]
    return _lib.RULE_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        0 if a_log is None else a_log.data_ptr(), 0 if dt_bias is None else dt_bias.data_ptr(),
        states.data_ptr(), 0 if query_start_loc is None else query_start_loc.data_ptr(),
        cache_indices.data_ptr(), 0 if has_initial_state is None else has_initial_state.data_ptr(),
        out.data_ptr(),
        tokens, num_seqs, heads, qk_heads, dim,
        qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
        gs[0], gs[1], 1 if per_channel else 0, bs[0], bs[1],
        states.shape[0], ss[0], ss[1], cache_indices.stride()[0],
        0 if null_block_id is None else int(null_block_id),
        dim ** -0.5 if scale is None else float(scale), L2_EPS if qk_l2norm else -1.0,
        0.0 if lower_bound is None else float(lower_bound),
        code, DTYPE_CODES[g.dtype], DTYPE_CODES[beta.dtype], gate, int(beta_logits),
        int(null_block_id is not None))


def _output(v, out):
    if out is None:
        return _fresh_like(v)
    if (out.shape != v.shape or out.dtype != v.dtype or not out.is_contiguous()
            or out.get_device() != v.get_device()):
        raise ValueError(f"out must be a contiguous {v.dtype} tensor of shape {tuple(v.shape)} on {v.device}")
    return out


def gated_delta_rule_fn(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    beta: torch.Tensor,
    states: torch.Tensor,
    query_start_loc: torch.Tensor,
    cache_indices: torch.Tensor,
    has_initial_state: Optional[torch.Tensor],
    *,
    a_log: Optional[torch.Tensor] = None,
    dt_bias: Optional[torch.Tensor] = None,
    lower_bound: Optional[float] = None,
    beta_logits: bool = False,
    qk_l2norm: bool = True,
    scale: Optional[float] = None,
    null_block_id: Optional[int] = NULL_BLOCK_ID,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """The gated delta rule over packed sequences (prefill).

    For every token t of a sequence and every head, with a state S of (key channel, value
    channel)::

        S = diag(exp(log_decay_t)) S
        S = S + k_t beta_t (v_t - S^T k_t)^T
        out_t = scale * S^T q_t

    q, k (tokens, qk heads, head_dim) and v (tokens, heads, head_dim) are bfloat16, float16 or
    float32 with a contiguous last axis: a plane of ``packed_causal_conv1d_fn``, viewed as
    (tokens, heads, head_dim), is one of them. head_dim is 64 or 128; heads is a multiple of
    qk heads, and value head h uses query and key head h // (heads // qk heads). With
    ``qk_l2norm`` q and k are divided by sqrt(|.|^2 + 1e-6) first. scale defaults to
    head_dim ** -0.5.

    g (tokens, heads, head_dim), or (tokens, heads) for one gate per head, is in v's dtype or
    float32. It is the log decay itself (at most 0), or with ``a_log`` (heads,) the gate's input::

        -exp(a_log) * softplus(g + dt_bias)                      # lower_bound None
        lower_bound * sigmoid(exp(a_log) * (g + dt_bias))        # otherwise

    with dt_bias (heads, head_dim) float32 or None. beta (tokens, heads) is the step size, or
    with ``beta_logits`` its logit.

    states (cache lines, heads, head_dim, head_dim) float32 is read and written in place.
    query_start_loc, cache_indices, has_initial_state and null_block_id mean what they mean
    for ``packed_causal_conv1d_fn``; rows no sequence owns are left unwritten, and a sequence
    without tokens leaves what it starts from (zeros in its line without an initial state, where
    ``packed_causal_conv1d_fn`` leaves its line alone). A value that is not finite reaches no
    earlier token. Returns (tokens, heads, head_dim) in v's dtype (``out``, when given; it may not
    overlap an input). The state and every intermediate hold FP32 or 22-bit pairs; only the output
    is rounded to its dtype. Takes about 60 KB of scratch memory per 32 tokens and head of 128 from
    torch's allocator (16 GB for 131072 tokens of 64 heads). Queued on the current stream; no
    synchronisation.
    """
    sizes = _heads(q, k, v, g, beta, states)
    out = _output(v, out)
    if query_start_loc.dtype != torch.int32 or query_start_loc.dim() != 1 or not query_start_loc.is_contiguous():
        raise ValueError("query_start_loc must be a contiguous 1-D int32 tensor")
    num_seqs = query_start_loc.shape[0] - 1
    if sizes[0] == 0 or num_seqs <= 0 or sizes[1] == 0:
        return out
    if has_initial_state is not None and (
            has_initial_state.dtype not in _FLAGS or not has_initial_state.is_contiguous()
            or has_initial_state.numel() < num_seqs):
        raise ValueError("has_initial_state must be a contiguous bool tensor with one entry per "
                         "sequence, or None")
    args = _pack(q, k, v, g, beta, states, cache_indices, query_start_loc, has_initial_state,
                 num_seqs, sizes, a_log, dt_bias, lower_bound, beta_logits, qk_l2norm, scale,
                 null_block_id, out)
    lib = _lib.load()
    need = lib.kdaconv_gated_delta_rule_workspace(sizes[0], num_seqs, sizes[1], sizes[3])
    # Memory of the current stream: the allocator hands it out again only to work that is
    # queued behind this call.
    scratch = torch.empty(need, dtype=torch.uint8, device=v.device) if need > 0 else None
    rc = _call(v.get_device(), lib.kdaconv_gated_delta_rule, args,
               None if scratch is None else scratch.data_ptr(), need)
    _lib.check(rc, "gated_delta_rule_fn")
    return out


def gated_delta_rule_update(
    q: torch.Tensor,
    k: torch.Tensor,
    v: torch.Tensor,
    g: torch.Tensor,
    beta: torch.Tensor,
    states: torch.Tensor,
    cache_indices: torch.Tensor,
    *,
    a_log: Optional[torch.Tensor] = None,
    dt_bias: Optional[torch.Tensor] = None,
    lower_bound: Optional[float] = None,
    beta_logits: bool = False,
    qk_l2norm: bool = True,
    scale: Optional[float] = None,
    null_block_id: Optional[int] = NULL_BLOCK_ID,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Decode step of ``gated_delta_rule_fn``: row b of q, k, v, g and beta is the one token
    of sequence b, which continues from states[cache_indices[b]] (zeros for the null block,
    whose line is neither read nor written). Arguments and result as there."""
    sizes = _heads(q, k, v, g, beta, states)
    out = _output(v, out)
    if sizes[0] == 0 or sizes[1] == 0:
        return out
    args = _pack(q, k, v, g, beta, states, cache_indices, None, None, sizes[0], sizes, a_log,
                 dt_bias, lower_bound, beta_logits, qk_l2norm, scale, null_block_id, out)
    rc = _call(v.get_device(), _lib.load().kdaconv_gated_delta_rule_update, args)
    _lib.check(rc, "gated_delta_rule_update")
    return out


def gated_delta_rule_supported(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                               beta: torch.Tensor, states: torch.Tensor) -> bool:
    """Whether gated_delta_rule_fn serves these tensors, and gated_delta_rule_update their rows
    (of up to 2^23 sequences times heads)."""
    try:
        sizes = _heads(q, k, v, g, beta, states)
        lib = _lib.load()
        one = torch.empty(2, dtype=torch.int32, device=v.device)
        # As one sequence. The output and the scratch memory would be fresh allocations: v and any
        # aligned address stand in for them.
        args = _pack(q, k, v, g, beta, states, one, one, None, 1, sizes, None, None, None,
                     False, True, None, None, v)
    except (ValueError, _lib.LibraryMissing):
        return False
    return lib.kdaconv_gated_delta_rule_validate(args, 0, 256, 1 << 62) == _lib.OK
