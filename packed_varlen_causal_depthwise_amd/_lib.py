"""ctypes binding of libkdaconv (include/kdaconv.h). Argument marshalling only."""

from __future__ import annotations

import ctypes
import pathlib
import struct

LIBRARY = pathlib.Path(__file__).resolve().parent / "libkdaconv.so"

OK, EINVAL, EUNSUPPORTED, ELAUNCH = 0, 1, 2, 3
ACT_NONE, ACT_SILU = 0, 1
BF16, F16, F32 = 0, 1, 2
GATE_LOG, GATE_SOFTPLUS, GATE_BOUNDED = 0, 1, 2
NORM_GATE_NONE, NORM_GATE_SIGMOID, NORM_GATE_SILU = 0, 1, 2

#: kdaconv_rule_args: 12 pointers, 21 integers, 3 doubles, 6 32-bit integers, no padding.
RULE_ARGS = struct.Struct("=12Q21q3d6i")

#: kdaconv_latent_cache: 3 pointers, 10 integers, 2 32-bit integers, no padding.
LATENT_CACHE = struct.Struct("=3Q10q2i")
#: kdaconv_latent_args after its cache: 6 pointers, 9 integers, 1 double.
LATENT_ARGS = struct.Struct("=6Q9qd")
#: kdaconv_expanded_args: 7 pointers, 14 integers, 1 double, 2 32-bit integers, no padding.
EXPANDED_ARGS = struct.Struct("=7Q14qd2i")

# Every entry point include/kdaconv.h declares.
EXPORTS = (
    "kdaconv_packed_causal_conv1d",
    "kdaconv_packed_causal_conv1d_update",
    "kdaconv_packed_causal_conv1d_update_bf16_state",
    "kdaconv_validate",
    "kdaconv_activation_map",
    "kdaconv_gated_delta_rule",
    "kdaconv_gated_delta_rule_update",
    "kdaconv_gated_delta_rule_validate",
    "kdaconv_gated_delta_rule_workspace",
    "kdaconv_gated_rms_norm",
    "kdaconv_residual_rms_norm",
    "kdaconv_rotary_embedding",
    "kdaconv_latent_cache_write",
    "kdaconv_latent_cache_read",
    "kdaconv_latent_attention",
    "kdaconv_latent_attention_update",
    "kdaconv_latent_attention_validate",
    "kdaconv_latent_attention_workspace",
    "kdaconv_expanded_attention",
    "kdaconv_expanded_attention_validate",
    "kdaconv_expanded_attention_workspace",
    "kdaconv_status_string",
    "kdaconv_version",
)

_lib = None


class LibraryMissing(ImportError):
    pass


def load() -> ctypes.CDLL:
    """Load libkdaconv.so from the package directory; raise if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIBRARY.exists():
        raise LibraryMissing(
            f"{LIBRARY} is missing: build it with `python -m packed_varlen_causal_depthwise_amd.build`"
            " (or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(str(LIBRARY))
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    conv_args = [
        vp, i32, i64, i64, i64,  # x, dtype, num_tokens, dim, x_row_stride
        vp, i64, i64, vp,  # weight, weight strides, bias
        vp, i64, i64, i64, i64,  # conv_states, num_cache_lines, strides
        vp, i64,  # query_start_loc, num_seqs
        vp, i64, vp,  # cache_indices, stride, has_initial_state
        i64, i32, i32, i64,  # part_dim, activation, has_null_block, null_block_id
        vp,  # out
    ]
    lib.kdaconv_packed_causal_conv1d.argtypes = conv_args + [vp]
    lib.kdaconv_packed_causal_conv1d.restype = i32
    lib.kdaconv_packed_causal_conv1d_update.argtypes = [
        vp, i32, i64, i64, i64,  # x, dtype, batch, dim, x_row_stride
        vp, i64, i64, vp,  # weight, weight strides, bias
        vp, i64, i64, i64, i64,  # conv_states, num_cache_lines, strides
        vp, i64,  # cache_indices, stride
        i64, i32, i32, i64,  # part_dim, activation, has_null_block, null_block_id
        vp, vp,  # out, stream
    ]
    lib.kdaconv_packed_causal_conv1d_update.restype = i32
    lib.kdaconv_packed_causal_conv1d_update_bf16_state.argtypes = [
        vp, i32, i64, i64, i64,  # x, dtype, batch, dim, x_row_stride
        vp, i64, i64, i64, vp,  # weight, part stride, channel stride, width stride, bias
        vp, i64, i64, i64, i64,  # conv_states (bf16), num_cache_lines, strides
        vp, i64,  # cache_indices, stride
        i64, i32, i32, i64,  # part_dim, activation, has_null_block, null_block_id
        vp, vp,  # out, stream
    ]
    lib.kdaconv_packed_causal_conv1d_update_bf16_state.restype = i32
    lib.kdaconv_validate.argtypes = conv_args
    lib.kdaconv_validate.restype = i32
    lib.kdaconv_activation_map.argtypes = [ctypes.c_uint32, i64, i32, i32, vp, vp]
    lib.kdaconv_activation_map.restype = i32
    # The argument struct is passed as the bytes RULE_ARGS packs.
    packed, f64 = ctypes.c_char_p, ctypes.c_double
    lib.kdaconv_gated_delta_rule.argtypes = [packed, vp, i64, vp]
    lib.kdaconv_gated_delta_rule.restype = i32
    lib.kdaconv_gated_delta_rule_update.argtypes = [packed, vp]
    lib.kdaconv_gated_delta_rule_update.restype = i32
    lib.kdaconv_gated_delta_rule_validate.argtypes = [packed, i32, vp, i64]
    lib.kdaconv_gated_delta_rule_validate.restype = i32
    lib.kdaconv_gated_delta_rule_workspace.argtypes = [i64, i64, i64, i64]
    lib.kdaconv_gated_delta_rule_workspace.restype = i64
    lib.kdaconv_gated_rms_norm.argtypes = [
        vp, i32, i64, i64, i64, i64, i64,  # x, dtype, tokens, heads, dim, x strides
        vp, i64, i64, i32,  # gate, strides, activation
        vp, f64, vp, vp,  # weight, eps, out, stream
    ]
    lib.kdaconv_gated_rms_norm.restype = i32
    lib.kdaconv_residual_rms_norm.argtypes = [
        vp, i32, i64, i64, i64,  # x, dtype, tokens, hidden, x stride
        vp, i64, f64,  # residual, stride, scale
        vp, f64, vp, vp,  # weight, eps, out, stream
    ]
    lib.kdaconv_residual_rms_norm.restype = i32
    lib.kdaconv_rotary_embedding.argtypes = [
        vp, i32, i64, i64, i64, i64, i64,  # x, dtype, tokens, heads, dim, x strides
        vp, i32, vp, i64, i64, i32, f64,  # positions, 64 bits, inv_freq, rotary, offset, interleaved, scale
        vp, i64, i64, vp,  # out, strides, stream
    ]
    lib.kdaconv_rotary_embedding.restype = i32
    lib.kdaconv_latent_cache_write.argtypes = [
        packed, vp, i64, vp, i64, i64,  # cache, latent, stride, rope, stride, tokens
        vp, i32, vp, f64,  # slots, 64 bits, weight, eps
        vp, i32, vp, i32, f64, vp,  # positions, 64 bits, inv_freq, interleaved, scale, stream
    ]
    lib.kdaconv_latent_cache_write.restype = i32
    lib.kdaconv_latent_cache_read.argtypes = [
        packed, vp, i64, i64,  # cache, block_table, stride, pages per sequence
        vp, i64, i64, vp, vp,  # kv_start_loc, num_seqs, num_tokens, out, stream
    ]
    lib.kdaconv_latent_cache_read.restype = i32
    for name in ("kdaconv_latent_attention", "kdaconv_latent_attention_update"):
        getattr(lib, name).argtypes = [packed, vp, i64, vp]
        getattr(lib, name).restype = i32
    lib.kdaconv_latent_attention_validate.argtypes = [packed, i32, vp, i64]
    lib.kdaconv_latent_attention_validate.restype = i32
    lib.kdaconv_latent_attention_workspace.argtypes = [i64, i64, i64, i64]
    lib.kdaconv_latent_attention_workspace.restype = i64
    lib.kdaconv_expanded_attention.argtypes = [packed, vp, i64, vp]
    lib.kdaconv_expanded_attention.restype = i32
    lib.kdaconv_expanded_attention_workspace.argtypes = [i64, i64, i64, i64, i64]
    lib.kdaconv_expanded_attention_workspace.restype = i64
    lib.kdaconv_expanded_attention_validate.argtypes = [packed, vp, i64]
    lib.kdaconv_expanded_attention_validate.restype = i32
    lib.kdaconv_status_string.argtypes = [i32]
    lib.kdaconv_status_string.restype = ctypes.c_char_p
    lib.kdaconv_version.argtypes = []
    lib.kdaconv_version.restype = i32
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().kdaconv_status_string(code).decode()


def check(code: int, what: str) -> None:
    if code == OK:
        return
    msg = f"{what}: {status_string(code)} (status {code})"
    if code in (EINVAL, EUNSUPPORTED):
        raise ValueError(msg)
    raise RuntimeError(msg)
