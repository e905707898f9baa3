"""A KDA attention layer out of this library's operators: prefill of packed prompts, then
decoding, over one paged cache.

    python examples/kda_layer.py [--prompts 3] [--tokens 900] [--steps 8] [--dtype bf16]

Per call: residual_rms_norm -> input projection -> packed_causal_conv1d (q, k and v) ->
gated_delta_rule (decay gate and step size straight from the projection's rows) ->
gated_rms_norm -> output projection. The two projections are plain library products. All
weights are random; the command prints what the layer did and how far decoding is from
prefilling the same tokens.
"""

from __future__ import annotations

import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))

import packed_varlen_causal_depthwise_amd as kd  # noqa: E402


class KdaLayer:
    """One layer and its cache: a conv state and a delta-rule state per cache line."""

    EPS = 1e-5

    def __init__(self, heads=4, head_dim=128, hidden=512, lines=8, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=gen) * scale

        self.heads, self.head_dim, self.part = heads, head_dim, heads * head_dim
        part, dev = self.part, dict(device=device)
        # Columns: q | k | v | decay gate | output gate | step size logits, padded to 64.
        self.width = 5 * part + (heads + 63) // 64 * 64
        self.in_proj = normal(hidden, self.width, scale=hidden ** -0.5).to(dtype).to(**dev)
        self.out_proj = normal(part, hidden, scale=part ** -0.5).to(dtype).to(**dev)
        self.conv_weight = normal(3 * part, 4, scale=0.5).to(**dev)
        self.norm_weight = (1 + 0.1 * normal(hidden)).to(**dev)
        self.head_weight = (1 + 0.1 * normal(head_dim)).to(**dev)
        self.a_log = (torch.rand(heads, generator=gen) * 2.0).to(**dev)
        self.dt_bias = (normal(heads, head_dim) - 3.0).to(**dev)
        self.conv_states = torch.zeros(lines, 3 * part, 3, **dev)
        self.states = torch.zeros(lines, heads, head_dim, head_dim, **dev)

    def _columns(self, rows):
        """The projection's pieces, as views of its rows."""
        n, part, heads, dim = rows.shape[0], self.part, self.heads, self.head_dim
        gate = rows[:, 3 * part:4 * part].view(n, heads, dim)
        out_gate = rows[:, 4 * part:5 * part].view(n, heads, dim)
        return rows[:, :3 * part], gate, out_gate, rows[:, 5 * part:5 * part + heads]

    def _rule(self, planes, gate, beta):
        n = planes.shape[1]
        q, k, v = planes.view(3, n, self.heads, self.head_dim)
        return (q, k, v, gate, beta, self.states), dict(
            a_log=self.a_log, dt_bias=self.dt_bias, lower_bound=-5.0, beta_logits=True,
            null_block_id=None)

    def _finish(self, o, out_gate):
        o = kd.gated_rms_norm(o, out_gate, self.head_weight, eps=self.EPS)
        return o.view(o.shape[0], self.part) @ self.out_proj

    def prefill(self, x, residual, query_start_loc, cache_indices, has_initial_state):
        """The layer's output for packed sequences; residual takes x in place."""
        rows = kd.residual_rms_norm(x, residual, self.norm_weight, eps=self.EPS) @ self.in_proj
        qkv, gate, out_gate, beta = self._columns(rows)
        planes = kd.packed_causal_conv1d_fn(
            qkv, self.conv_weight, None, self.conv_states, query_start_loc, cache_indices,
            has_initial_state, self.part, activation="silu", null_block_id=None)
        args, kw = self._rule(planes, gate, beta)
        o = kd.gated_delta_rule_fn(*args, query_start_loc, cache_indices, has_initial_state, **kw)
        return self._finish(o, out_gate)

    def decode(self, x, residual, cache_indices):
        """One token per sequence, continuing from the cache."""
        rows = kd.residual_rms_norm(x, residual, self.norm_weight, eps=self.EPS) @ self.in_proj
        qkv, gate, out_gate, beta = self._columns(rows)
        planes = kd.packed_causal_conv1d_update(
            qkv, self.conv_weight, None, self.conv_states, cache_indices, self.part,
            activation="silu", null_block_id=None)
        args, kw = self._rule(planes, gate, beta)
        o = kd.gated_delta_rule_update(*args, cache_indices, **kw)
        return self._finish(o, out_gate)


def lengths_of(prompts, tokens):
    """Prompt lengths about tokens / prompts, all different."""
    base = max(1, tokens // prompts)
    return [max(1, base + (7 * i) % 13 - 6) for i in range(prompts)]


def compare(prompts=3, tokens=900, steps=8, dtype=torch.bfloat16, heads=4, head_dim=128, seed=0):
    """Prefills every prompt and decodes `steps` tokens after it; prefills the same tokens in
    one go on other cache lines. Returns the last tokens' outputs both ways, and the layer."""
    layer = KdaLayer(heads, head_dim, lines=2 * prompts, dtype=dtype, seed=seed)
    hidden = layer.in_proj.shape[0]
    lengths = lengths_of(prompts, tokens)
    gen = torch.Generator().manual_seed(seed + 1)
    x = [torch.randn(n + steps, hidden, generator=gen).to(dtype).cuda() for n in lengths]

    def starts(ns):
        return torch.tensor([0] + ns, device="cuda").cumsum(0).to(torch.int32)

    new = torch.zeros(prompts, dtype=torch.bool, device="cuda")
    lines = torch.arange(prompts, dtype=torch.int32, device="cuda")
    packed = torch.cat([t[:n] for t, n in zip(x, lengths)])
    layer.prefill(packed, torch.zeros_like(packed), starts(lengths), lines, new)
    for i in range(steps):
        tok = torch.stack([t[n + i] for t, n in zip(x, lengths)])
        stepped = layer.decode(tok, torch.zeros_like(tok), lines)

    whole = torch.cat(x)
    ends = starts([n + steps for n in lengths])
    out = layer.prefill(whole, torch.zeros_like(whole), ends, lines + prompts, new)
    return stepped, out[ends[1:].long() - 1], layer


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--prompts", type=int, default=3)
    p.add_argument("--tokens", type=int, default=900, help="prompt tokens in all")
    p.add_argument("--steps", type=int, default=8, help="tokens decoded after each prompt")
    p.add_argument("--dtype", choices=["bf16", "fp16", "fp32"], default="bf16")
    a = p.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[a.dtype]
    stepped, whole, layer = compare(a.prompts, a.tokens, a.steps, dtype)
    n = a.prompts
    state = (layer.states[:n] - layer.states[n:]).norm() / layer.states[n:].norm()
    last = (stepped.float() - whole.float()).norm() / whole.float().norm()
    print(f"{n} prompts of {lengths_of(n, a.tokens)} tokens, {a.steps} decode steps, {a.dtype}")
    print(f"decode against prefill of the same tokens: last outputs {last.item():.2e}, "
          f"states {state.item():.2e} (relative)")


if __name__ == "__main__":
    main()
