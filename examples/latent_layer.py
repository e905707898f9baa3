"""A latent attention layer out of this library's operators, to stand between KDA layers:
prefill of packed prompts in chunks, then decoding, over one paged cache.

    python examples/latent_layer.py [--prompts 3] [--tokens 900] [--steps 8] [--dtype bf16] [--cache same]

Per call: residual_rms_norm -> input projection -> rotary_embedding (the queries) ->
latent_cache_write (norms the latents, turns their rotated part) -> attention -> output
projection. First chunks of prompts attend in the expanded form, with keys and values from the
up-projection; later chunks too, with the earlier tokens out of latent_cache_read; decode steps
and short chunks in the absorbed form over the cache itself. The projections are plain library
products. All weights are random; the command prints how far the ways are apart.
"""

from __future__ import annotations

import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))

import packed_varlen_causal_depthwise_amd as kd  # noqa: E402


def starts(lengths, device="cuda"):
    return torch.tensor([0] + list(lengths), device=device).cumsum(0).to(torch.int32)


class LatentLayer:
    """One layer and its paged cache."""

    EPS = 1e-6

    def __init__(self, heads=4, head_dim=128, rope_dim=64, latent=512, hidden=512, pages=64, page_size=64,
                 dtype=torch.bfloat16, e4m3=False, factor=1.0, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(device)

        self.heads, self.head_dim, self.rope_dim, self.latent = heads, head_dim, rope_dim, latent
        self.query = heads * (head_dim + rope_dim)
        # Columns: the queries | the latent | the part to rotate.
        self.in_proj = normal(hidden, self.query + latent + rope_dim, scale=hidden ** -0.5)
        # Per head the latent's keys, then its values.
        self.up_proj = normal(latent, heads * 2 * head_dim, scale=latent ** -0.5)
        up = self.up_proj.view(latent, heads, 2, head_dim)
        self.up_keys = up[:, :, 0].permute(1, 2, 0).contiguous()  # (heads, head_dim, latent)
        self.up_values = up[:, :, 1].permute(1, 0, 2).contiguous()  # (heads, latent, head_dim)
        self.out_proj = normal(heads * head_dim, hidden, scale=(heads * head_dim) ** -0.5)
        self.norm_weight = (1 + 0.1 * torch.randn(hidden, generator=gen)).to(device)
        self.latent_weight = (1 + 0.1 * torch.randn(latent, generator=gen)).to(device)
        # The factor of a stretched context is one on queries and on keys, all of their channels: it
        # goes into the scale, for only a part of a head is turned.
        self.inv_freq, temper = kd.rotary_frequencies(rope_dim, factor=factor, device=device)
        self.scale = (head_dim + rope_dim) ** -0.5 * temper ** 2
        self.ropes = torch.zeros(pages, page_size, rope_dim, dtype=dtype, device=device)
        kind = torch.float8_e4m3fn if e4m3 else dtype
        self.latents = torch.zeros(pages, page_size, latent, dtype=dtype, device=device).to(kind)
        self.scales = torch.zeros(pages, page_size, latent // 32, dtype=torch.uint8, device=device) if e4m3 else None

    @property
    def cache(self):
        return self.latents, self.ropes, self.scales

    def slots(self, table, seqs, positions):
        """Places in the cache of tokens `positions` of sequences `seqs`."""
        page = self.ropes.shape[1]
        return table[seqs, positions // page].long() * page + positions % page

    def _into_cache(self, x, residual, positions, slots):
        """The queries, turned; the tokens' latents go into the cache."""
        rows = kd.residual_rms_norm(x, residual, self.norm_weight, eps=self.EPS) @ self.in_proj
        q = rows[:, :self.query].view(-1, self.heads, self.head_dim + self.rope_dim)
        latent, rope = rows[:, self.query:].split([self.latent, self.rope_dim], 1)
        kd.rotary_embedding(q, positions, self.inv_freq, offset=self.head_dim, out=q)
        kd.latent_cache_write(latent, rope, *self.cache, slots, weight=self.latent_weight, eps=self.EPS,
                              positions=positions, inv_freq=self.inv_freq)
        return q

    def _absorbed(self, q):
        """The queries times the keys' up-projection, head by head."""
        return torch.bmm(q[..., :self.head_dim].transpose(0, 1).contiguous(), self.up_keys).transpose(0, 1)

    def _values(self, o):
        o = torch.bmm(o.transpose(0, 1).contiguous(), self.up_values).transpose(0, 1)
        return o.flatten(1) @ self.out_proj

    def prefill(self, x, residual, positions, slots, table, query_start_loc, kv_start_loc, num_keys):
        """Packed chunks of prompts in the expanded form. Sequence s has kv_start_loc's number of
        tokens, its chunk the last of them, num_keys in all."""
        q = self._into_cache(x, residual, positions, slots)
        kv = kd.latent_cache_read(*self.cache, table, kv_start_loc, num_keys)
        up = (kv[:, :self.latent] @ self.up_proj).view(num_keys, self.heads, 2 * self.head_dim)
        o = kd.expanded_attention_fn(q, up[..., :self.head_dim], kv[:, self.latent:], up[..., self.head_dim:],
                                     query_start_loc, kv_start_loc, scale=self.scale)
        return o.flatten(1) @ self.out_proj

    def extend(self, x, residual, positions, slots, table, lengths, query_start_loc):
        """Packed short chunks in the absorbed form; `lengths` counts their tokens already."""
        q = self._into_cache(x, residual, positions, slots)
        o = kd.latent_attention_fn(self._absorbed(q), q[..., self.head_dim:], *self.cache, table, lengths,
                                   query_start_loc, scale=self.scale)
        return self._values(o)

    def decode(self, x, residual, positions, slots, table, lengths):
        """One token per sequence."""
        q = self._into_cache(x, residual, positions, slots)
        o = kd.latent_attention_update(self._absorbed(q), q[..., self.head_dim:], *self.cache, table, lengths,
                                       scale=self.scale)
        return self._values(o)


def lengths_of(prompts, tokens):
    """Prompt lengths about tokens / prompts, all different."""
    base = max(1, tokens // prompts)
    return [max(1, base + (7 * i) % 13 - 6) for i in range(prompts)]


def compare(prompts=3, tokens=900, steps=8, dtype=torch.bfloat16, heads=4, head_dim=128, rope_dim=64, latent=512,
            page_size=64, e4m3=False, factor=1.0, seed=0):
    """Every prompt in two chunks (expanded), a short chunk (absorbed), then `steps` decode steps;
    then the same tokens in one expanded prefill on other pages. Returns the last tokens' outputs
    both ways, and the layer."""
    lengths = lengths_of(prompts, tokens)
    total = [n + steps for n in lengths]
    per = [-(-n // page_size) for n in total]
    layer = LatentLayer(heads, head_dim, rope_dim, latent, pages=2 * sum(per), page_size=page_size, dtype=dtype,
                        e4m3=e4m3, factor=factor, seed=seed)
    hidden = layer.in_proj.shape[0]
    gen = torch.Generator().manual_seed(seed + 1)
    x = [torch.randn(n, hidden, generator=gen).to(dtype).cuda() for n in total]
    order = torch.randperm(2 * sum(per), generator=gen).to(torch.int32)
    tables, first = torch.zeros(2, prompts, max(per), dtype=torch.int32), 0
    for one in tables:
        for s, n in enumerate(per):
            one[s, :n] = order[first:first + n]
            first += n
    tables = tables.cuda()

    def chunk(begin, end):
        """Packed tokens begin[s] .. end[s] of every sequence, and where they go."""
        seqs = torch.cat([torch.full((b - a,), s) for s, (a, b) in enumerate(zip(begin, end))]).cuda()
        positions = torch.cat([torch.arange(a, b) for a, b in zip(begin, end)]).cuda()
        rows = torch.cat([t[a:b] for t, a, b in zip(x, begin, end)])
        return rows, torch.zeros_like(rows), positions, seqs

    def prefill(table, begin, end):
        rows, residual, positions, seqs = chunk(begin, end)
        return layer.prefill(rows, residual, positions, layer.slots(table, seqs, positions), table,
                             starts([b - a for a, b in zip(begin, end)]), starts(end), sum(end))

    zero, half = [0] * prompts, [n // 2 for n in lengths]
    short = [max(h, n - 3) for h, n in zip(half, lengths)]
    table = tables[0]
    prefill(table, zero, half)
    prefill(table, half, short)
    rows, residual, positions, seqs = chunk(short, lengths)
    stepped = layer.extend(rows, residual, positions, layer.slots(table, seqs, positions), table,
                           torch.tensor(lengths, dtype=torch.int32).cuda(),
                           starts([b - a for a, b in zip(short, lengths)]))
    stepped = stepped[starts([b - a for a, b in zip(short, lengths)])[1:].long() - 1]
    for i in range(steps):
        rows, residual, positions, seqs = chunk([n + i for n in lengths], [n + i + 1 for n in lengths])
        stepped = layer.decode(rows, residual, positions, layer.slots(table, seqs, positions), table,
                               (positions + 1).to(torch.int32))
    out = prefill(tables[1], zero, total)
    return stepped, out[starts(total)[1:].long() - 1], layer


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--prompts", type=int, default=3)
    p.add_argument("--tokens", type=int, default=900, help="prompt tokens in all")
    p.add_argument("--steps", type=int, default=8, help="tokens decoded after each prompt")
    p.add_argument("--dtype", choices=["bf16", "fp16"], default="bf16")
    p.add_argument("--cache", choices=["same", "e4m3"], default="same", help="the latents' type in the cache")
    a = p.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[a.dtype]
    stepped, whole, _ = compare(a.prompts, a.tokens, a.steps, dtype, e4m3=a.cache == "e4m3")
    last = (stepped.float() - whole.float()).norm() / whole.float().norm()
    print(f"{a.prompts} prompts of {lengths_of(a.prompts, a.tokens)} tokens, {a.steps} decode steps, {a.dtype}, "
          f"cache {a.cache}")
    print(f"chunks and decode steps against one prefill of the same tokens: last outputs {last.item():.2e} (relative)")


if __name__ == "__main__":
    main()
