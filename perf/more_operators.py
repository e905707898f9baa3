"""Cases and plain forms of latent attention and of the cache and rotation it works with.

The cases stand for the attention layer that alternates with KDA layers in a hybrid model, whose
keys and values all come from one latent vector and one rotated vector a token:

- ``rotary``: rotary positions on the rotated part of the queries, in place.
- ``write``: the norm, the rotation and the store of new tokens into the paged cache.
- ``refill``: the same into an 8-bit cache, and the read of all the sequences' tokens back out
  of it (what a prompt's next chunk does before its keys and values are expanded).
- ``decode``: one token per sequence over the paged cache (absorbed form).
- ``chunk``: some new tokens per sequence over the paged cache (absorbed form).
- ``expanded``: packed prompts, with keys and values expanded for every head.

``run`` computes a case's operator in its plain form where ``own`` is false, and makes the package's
calls where it is true. The plain forms work in FP32, the rotation's angles and the norm in FP64:
the first are far from zero, the second ends next to rounding borders of the 8-bit cache.
``exact`` evaluates the definitions in FP64.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NORM_EPS = 1e-6
#: Channels of a latent that share one scale in the 8-bit cache.
BLOCK = 32


# ---------------------------------------------------------------------------- cases


def _rotary(name, tokens, heads, dim, rotary, interleaved, factor, dtype):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "factor": factor, "dtype": dtype}


def _write(name, tokens, latent, rope, page, dtype):
    return {"name": name, "op": "write", "tokens": tokens, "latent": latent, "rope": rope,
            "page": page, "interleaved": True, "dtype": dtype}


def _refill(name, seqs, tokens, cached, latent, rope, page, dtype):
    return {"name": name, "op": "refill", "seqs": seqs, "tokens": tokens, "cached": cached,
            "latent": latent, "rope": rope, "page": page, "interleaved": False, "dtype": dtype}


def _attend(name, op, seqs, tokens, cached, lengths, heads, latent, rope, page, cache, dtype):
    return {"name": name, "op": op, "seqs": seqs, "tokens": tokens, "cached": cached,
            "lengths": lengths, "heads": heads, "latent": latent, "rope": rope, "page": page,
            "cache": cache, "dtype": dtype}


def _expanded(name, seqs, tokens, cached, lengths, heads, dim, rope, dtype):
    return {"name": name, "op": "expanded", "seqs": seqs, "tokens": tokens, "cached": cached,
            "lengths": lengths, "heads": heads, "dim": dim, "rope": rope, "dtype": dtype}


def listed():
    return [
        # The queries of an ordinary decode batch, 12 heads of 128 + 64: latency counts.
        _rotary("rotary 37 tokens", 37, 12, 192, 64, True, 1.0, "bf16"),
        # A whole prefill budget, with a context stretched 32 times.
        _rotary("rotary 16384 tokens", 16384, 12, 192, 64, False, 32.0, "bf16"),
        # The new tokens of a decode batch go into the cache: the shortest call of the set.
        _write("write 37 tokens", 37, 512, 64, 64, "bf16"),
        # A whole prefill budget goes into the cache.
        _write("write 16384 tokens", 16384, 512, 64, 64, "bf16"),
        # The second chunks of a few prompts, odd lengths and small pages, fp16.
        _refill("refill 999 + 3005 tokens e4m3", 8, 999, 3005, 512, 64, 16, "f16"),
        # The last chunk of one very long prompt.
        _refill("refill 16384 + 114688 e4m3", 1, 16384, 114688, 512, 64, 64, "bf16"),
        # One sequence decodes over a long context: latency, and the split of one sequence.
        _attend("decode 1 sequence", "decode", 1, 1, 16000, "equal", 12, 512, 64, 64, "same", "bf16"),
        # An ordinary batch of very unequal contexts, 8-bit cache.
        _attend("decode 37 sequences e4m3", "decode", 37, 37, 90001, "lognormal", 12, 512, 64, 64,
                "e4m3", "bf16"),
        # A full serving batch: the cache's bytes, 1.2 GB.
        _attend("decode 256 sequences", "decode", 256, 256, 1048576, "uniform", 12, 512, 64, 64,
                "same", "bf16"),
        # Speculative steps and short prompts over contexts, 8 heads, small pages, fp16.
        _attend("chunk 24 sequences fp16", "chunk", 24, 500, 70007, "uniform", 8, 512, 64, 16,
                "same", "f16"),
        # A few short prompts scheduled together.
        _expanded("expanded 8 short prompts", 8, 1204, 0, "uniform", 12, 128, 64, "bf16"),
        # A whole prefill budget spent on one long prompt: matrix products.
        _expanded("expanded 16384 tokens", 1, 16384, 0, "equal", 12, 128, 64, "bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "refill", "decode", "decode", "decode", "chunk", "chunk",
                     "expanded", "expanded", "expanded"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rotary":
        rotary = rng.choice([32, 64, 128])
        heads = rng.randint(1, 32)
        most = min(16384, 16384 * 12 * 64 // (heads * rotary))
        return {"op": op, "tokens": _log_int(rng, 1, most), "heads": heads,
                "dim": rotary + rng.choice([0, 64, 128]), "rotary": rotary,
                "interleaved": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 32.0]),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    latent, rope = rng.choice([512, 512, 256, 384]), rng.choice([64, 64, 32])
    page = rng.choice([1, 16, 32, 48, 64, 128])
    if op == "write":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "latent": latent, "rope": rope,
                "page": page, "interleaved": rng.random() < 0.5, "dtype": dtype}
    if op == "refill":
        seqs = _log_int(rng, 1, 64)
        tokens = _log_int(rng, seqs, 16384)
        return {"op": op, "seqs": seqs, "tokens": tokens, "cached": rng.randint(0, 4 * tokens),
                "latent": latent, "rope": rope, "page": page,
                "interleaved": rng.random() < 0.5, "dtype": dtype}
    lengths = rng.choice(["equal", "uniform", "lognormal"])
    if op == "expanded":
        heads, dim = rng.choice([1, 3, 4, 8, 12, 16]), rng.choice([128, 128, 64])
        tokens = _log_int(rng, 1, 16384 * 12 // max(12, heads))
        seqs = _log_int(rng, 1, min(tokens, 64))
        # Contexts from earlier chunks, where the whole stays below the largest case.
        cached = rng.choice([0, rng.randint(0, 16384 - tokens) if tokens < 16384 else 0])
        return {"op": op, "seqs": seqs, "tokens": tokens, "cached": cached,
                "lengths": "uniform" if lengths == "lognormal" and seqs > 2 else lengths,
                "heads": heads, "dim": dim, "rope": rope, "dtype": dtype}
    cache = rng.choice(["same", "e4m3"])
    if op == "decode":
        seqs, heads = _log_int(rng, 1, 512), rng.choice([1, 4, 8, 12, 16, 32, 64])
        if lengths == "lognormal" and seqs > 128:  # the plain form pads to the longest
            lengths = "uniform"
        tokens = seqs
    else:
        seqs, heads = _log_int(rng, 1, 64), rng.choice([1, 4, 8, 12, 16])
        tokens = seqs * _log_int(rng, 1, 48)
    most = min(65536 * seqs, 1048576 * 12 // max(12, heads * tokens // seqs))
    return {"op": op, "seqs": seqs, "tokens": tokens, "cached": _log_int(rng, 1, most),
            "lengths": lengths, "heads": heads, "latent": latent, "rope": rope, "page": page,
            "cache": cache, "dtype": dtype}


# --------------------------------------------------------------------------- inputs


def _parts(total, count, kind, seed, least=0):
    """`count` host integers of at least `least` that sum to `total`."""
    g = torch.Generator().manual_seed(seed)
    if kind == "equal":
        w = torch.ones(count, dtype=torch.float64)
    elif kind == "uniform":
        w = torch.rand(count, generator=g, dtype=torch.float64) + 0.02
    else:
        w = torch.exp(torch.randn(count, generator=g, dtype=torch.float64))
    ends = torch.round(torch.cumsum(w, 0) / w.sum() * (total - least * count)).to(torch.int64)
    ends[-1] = total - least * count
    return [int(x) + least for x in torch.diff(ends, prepend=torch.zeros(1, dtype=torch.int64))]


def _starts(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _frequencies(rotary, factor):
    """Angles per position, a rotary base of 10000 and slow pairs stretched by the factor."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / rotary)
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * keep + f / factor * (1 - keep)).float().cuda()


def _pages(g, lengths, page, spare=3):
    """Pages of every sequence at random places: the table, the number of pages, and for each
    token of the packed sequences its slot."""
    per = [(n + page - 1) // page for n in lengths]
    count = sum(per) + spare
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + per, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(max(1, max(per)), device="cuda")[None]
    table = order[at.clamp(max=count - 1)]
    n = torch.tensor(lengths, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), n)
    pos = torch.arange(len(seq), device="cuda") - (torch.cumsum(n, 0) - n)[seq]
    slot = table[seq, pos // page].long() * page + pos % page
    return table, count, seq, pos, slot


def _cache(g, case, count, dtype, e4m3):
    """A cache of random tokens: latents, rotated parts, and scales of an 8-bit cache."""
    L, R, page = case["latent"], case["rope"], case["page"]
    if not e4m3:
        both = _normal(g, count, page, L + R).to(dtype)
        return both[..., :L], both[..., L:], None
    codes = (_normal(g, count, page, L) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.randint(118, 122, (count, page, (L + BLOCK - 1) // BLOCK), generator=g,
                           device="cuda").to(torch.uint8)
    return codes, _normal(g, count, page, R).to(dtype), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rotary":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        s["x"] = _normal(g, T, H, D).to(dt)
        s["positions"] = torch.randint(0, 131072, (T,), generator=g, device="cuda")
        s["inv_freq"] = _frequencies(case["rotary"], case["factor"])
        s["scale"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        return s
    if case["op"] in ("write", "refill"):
        L, R = case["latent"], case["rope"]
        T, page = case["tokens"], case["page"]
        e4m3 = case["op"] == "refill"
        if e4m3:
            new = _parts(T, case["seqs"], "uniform", seed * 31 + 1)
            old = _parts(case["cached"], case["seqs"], "uniform", seed * 31 + 2)
        else:
            new, old = [T], [0]
        table, count, seq, pos, slot = _pages(g, [a + b for a, b in zip(new, old)], page)
        before = torch.tensor(old, device="cuda")[seq]
        fresh = pos >= before
        s["slots"] = slot[fresh]
        s["positions"] = pos[fresh]
        s["latents"], s["ropes"], s["scales"] = _cache(g, case, count, dt, e4m3)
        # The projection's rows: the latent and the part to rotate, side by side.
        rows = _normal(g, T, L + R).to(dt)
        s["latent"], s["rope"] = rows[:, :L], rows[:, L:]
        s["weight"] = 1 + 0.1 * _normal(g, L)
        s["inv_freq"] = _frequencies(R, 1.0)
        s["block_table"], s["all_slots"], s["total"] = table, slot, len(seq)
        s["kv_start_loc"] = _starts([a + b for a, b in zip(new, old)])
        return s
    H = case["heads"]
    new = ([1] * case["seqs"] if case["op"] == "decode"
           else _parts(case["tokens"], case["seqs"], case["lengths"], seed * 31 + 1, least=1))
    old = _parts(case["cached"], case["seqs"], case["lengths"], seed * 31 + 2)
    lengths = [a + b for a, b in zip(new, old)]
    s["new"], s["lengths"] = new, lengths
    s["query_start_loc"] = _starts(new)
    T, S = case["tokens"], case["seqs"]
    # Padded places of queries and keys, for the plain form.
    n, m = torch.tensor(new, device="cuda"), torch.tensor(lengths, device="cuda")
    i = torch.arange(max(new), device="cuda")
    s["query_at"] = torch.where(i < n[:, None], s["query_start_loc"][:-1, None] + i, T)
    s["reach"] = (m - n)[:, None] + i + 1
    if case["op"] == "expanded":
        D, R, total = case["dim"], case["rope"], sum(lengths)
        s["q"] = _normal(g, T, H, D + R).to(dt)
        kv = _normal(g, total, H, 2 * D).to(dt)  # the up-projection's rows, key and value
        s["k"], s["v"] = kv[..., :D], kv[..., D:]
        s["k_rope"] = _normal(g, total, 512 + R).to(dt)[:, 512:]  # a slice of the cached rows
        s["kv_start_loc"] = _starts(lengths)
        j = torch.arange(max(lengths), device="cuda")
        s["key_at"] = torch.where(j < m[:, None], s["kv_start_loc"][:-1, None] + j, 0)
        s["scale"] = (D + R) ** -0.5
        return s
    L, R, page = case["latent"], case["rope"], case["page"]
    table, count, seq, pos, slot = _pages(g, lengths, page)
    s["latents"], s["ropes"], s["scales"] = _cache(g, case, count, dt, case["cache"] == "e4m3")
    s["block_table"], s["seq_lens"] = table, m.to(torch.int32)
    s["all_slots"] = slot
    j = torch.arange(max(lengths), device="cuda")
    j = torch.where(j < m[:, None], j, 0)
    s["key_at"] = table.gather(1, j // page).long() * page + j % page
    # Queries absorbed by a batched product over heads: head-major.
    s["q_latent"] = _normal(g, H, T, L).to(dt).transpose(0, 1)
    s["q_rope"] = _normal(g, T, H, 128 + R).to(dt)[..., 128:]
    s["scale"] = (128 + R) ** -0.5
    return s


# ---------------------------------------------------------------------- plain forms


def _turned(x, positions, inv_freq, interleaved, scale):
    """x (tokens, heads, rotary) in FP32, turned by the angles of the positions (FP64)."""
    a = positions.double()[:, None] * inv_freq.double()
    cos, sin = ((scale * f(a)).float()[:, None] for f in (torch.cos, torch.sin))
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    u, v = x.chunk(2, -1)
    return torch.cat([u * cos - v * sin, u * sin + v * cos], -1)


def _plain_rotary(s):
    part = s["x"][..., s["case"]["dim"] - s["case"]["rotary"]:]
    part.copy_(_turned(part.float(), s["positions"], s["inv_freq"], s["case"]["interleaved"], s["scale"]))
    return s["x"]


def _plain_write(s):
    case = s["case"]
    x = s["latent"].double()
    y = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * s["weight"].double()).float()
    r = _turned(s["rope"].float()[:, None], s["positions"], s["inv_freq"], case["interleaved"], 1.0)[:, 0]
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    s["ropes"][page, at] = r.to(s["ropes"].dtype)
    if s["scales"] is None:
        s["latents"][page, at] = y.to(s["latents"].dtype)
        return
    y = y.view(y.shape[0], -1, BLOCK)
    most = y.abs().amax(-1)
    e = torch.frexp(most / 448)[1]
    # frexp: most / 448 = m 2^e with m in [0.5, 1); m = 0.5 is a power of two itself
    e = torch.where(torch.ldexp(torch.full_like(most, 448.0), e - 1) >= most, e - 1, e).clamp(min=-100)
    codes = torch.ldexp(y, -e[..., None]).flatten(1).to(torch.float8_e4m3fn)
    s["latents"].view(torch.uint8)[page, at] = codes.view(torch.uint8)
    s["scales"][page, at] = (e + 127).to(torch.uint8)


def _rows(s, slots):
    """Latents and rotated parts of the slots, FP32."""
    page, at = slots // s["case"]["page"], slots % s["case"]["page"]
    r = s["ropes"][page, at].float()
    if s["scales"] is None:
        return s["latents"][page, at].float(), r
    c = s["latents"].view(torch.uint8)[page, at].view(torch.float8_e4m3fn).float()
    f = torch.exp2(s["scales"][page, at].float() - 127)
    return (c.unflatten(-1, (-1, BLOCK)) * f[..., None]).flatten(-2), r


def _plain_refill(s):
    _plain_write(s)
    return torch.cat(_rows(s, s["all_slots"]), -1).to(s["ropes"].dtype)


def _softmax_product(scores, reach, values):
    """Softmax over the keys below each query's reach, times the values."""
    below = torch.arange(scores.shape[-1], device=scores.device) < reach[..., None]
    scores = torch.where(below, scores, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - top)
    return (p @ values) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_attend(s):
    H, at = s["case"]["heads"], s["query_at"]
    S, n = at.shape
    q = torch.cat([s["q_latent"].float(), s["q_rope"].float()], -1)
    q = torch.cat([q, q[:1]])[at].flatten(1, 2)  # (seqs, n * heads, latent + rope)
    c, r = _rows(s, s["key_at"])
    scores = (q @ torch.cat([c, r], -1).transpose(1, 2)) * s["scale"]
    out = _softmax_product(scores, s["reach"].repeat_interleave(H, 1), c).unflatten(1, (n, H))
    dense = torch.empty(s["case"]["tokens"] + 1, H, c.shape[-1], dtype=s["q_latent"].dtype, device=c.device)
    dense[at] = out.to(dense.dtype)
    return dense[:-1]


def _plain_expanded(s):
    case, at, keys = s["case"], s["query_at"], s["key_at"]
    H, D, T = case["heads"], case["dim"], case["tokens"]
    q = torch.cat([s["q"], s["q"][:1]])[at].float().transpose(1, 2)  # (seqs, heads, n, dim)
    k = s["k"][keys].float().permute(0, 2, 3, 1)
    r = s["k_rope"][keys].float().transpose(1, 2)[:, None]
    scores = (q[..., :D] @ k + q[..., D:] @ r) * s["scale"]
    out = _softmax_product(scores, s["reach"][:, None], s["v"][keys].float().transpose(1, 2))
    dense = torch.empty(T + 1, H, D, dtype=s["q"].dtype, device=q.device)
    dense[at] = out.transpose(1, 2).to(dense.dtype)
    return dense[:T]


# ------------------------------------------------------------------- the package's calls


def _own(s):
    import packed_varlen_causal_depthwise_amd as kd

    case = s["case"]
    if case["op"] == "rotary":
        return kd.rotary_embedding(
            s["x"], s["positions"], s["inv_freq"], offset=case["dim"] - case["rotary"],
            interleaved=case["interleaved"], scale=s["scale"], out=s["x"])
    if case["op"] in ("write", "refill"):
        kd.latent_cache_write(
            s["latent"], s["rope"], s["latents"], s["ropes"], s["scales"], s["slots"],
            weight=s["weight"], eps=NORM_EPS, positions=s["positions"], inv_freq=s["inv_freq"],
            interleaved=case["interleaved"])
        if case["op"] == "write":
            return s["latents"], s["ropes"]
        return kd.latent_cache_read(s["latents"], s["ropes"], s["scales"], s["block_table"],
                                    s["kv_start_loc"], s["total"])
    if case["op"] == "decode":
        return kd.latent_attention_update(
            s["q_latent"], s["q_rope"], s["latents"], s["ropes"], s["scales"], s["block_table"],
            s["seq_lens"], scale=s["scale"])
    if case["op"] == "chunk":
        return kd.latent_attention_fn(
            s["q_latent"], s["q_rope"], s["latents"], s["ropes"], s["scales"], s["block_table"],
            s["seq_lens"], s["query_start_loc"], scale=s["scale"])
    return kd.expanded_attention_fn(s["q"], s["k"], s["k_rope"], s["v"], s["query_start_loc"],
                                    s["kv_start_loc"], scale=s["scale"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "write":
        _plain_write(state)
        return state["latents"], state["ropes"]
    return {"rotary": _plain_rotary, "refill": _plain_refill, "decode": _plain_attend,
            "chunk": _plain_attend, "expanded": _plain_expanded}[op](state)


# ------------------------------------------------------------------------ work and truth


def work(case):
    e, T = BYTES[case["dtype"]], case["tokens"]
    if case["op"] == "rotary":
        n = T * case["heads"] * case["rotary"]
        return {"bytes": 2 * e * n + 8 * T, "flops": 3 * n}
    if case["op"] == "expanded":
        H, D, R, total = case["heads"], case["dim"], case["rope"], T + case["cached"]
        pairs = T * (total - T / 2 + 0.5) / case["seqs"]  # of sequences of equal lengths
        return {"bytes": int(e * (T * H * (2 * D + R) + total * (2 * H * D + R))),
                "flops": int(2 * H * (2 * D + R) * pairs)}
    L, R = case["latent"], case["rope"]
    plain, eight = e * (L + R), L + e * R + L // BLOCK
    if case["op"] == "write":
        return {"bytes": T * (2 * plain + 16), "flops": 4 * T * (L + R)}
    if case["op"] == "refill":
        total = T + case["cached"]
        return {"bytes": T * (plain + eight + 16) + total * (eight + plain),
                "flops": 4 * T * (L + R) + total * L}
    H, total = case["heads"], T + case["cached"]
    row = eight if case["cache"] == "e4m3" else plain
    pairs = T * (total - T / 2 + 0.5) / case["seqs"]
    return {"bytes": int(total * row + e * T * H * (2 * L + R)), "flops": int(2 * H * (2 * L + R) * pairs)}


def _exact_turn(x, s, scale):
    a = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous())
    else:
        z = torch.complex(*x.chunk(2, -1))
    z = z * torch.polar(torch.full_like(a, scale), a)
    return torch.view_as_real(z).flatten(-2) if s["case"]["interleaved"] else torch.cat([z.real, z.imag], -1)


def _exact_codes(y):
    """What the 8-bit cache holds for y (tokens, latent), FP64: y in FP32, each block's largest
    value at most 448 steps of its power of two, four significant bits above 2^-6 of that."""
    y = y.float().double().unflatten(-1, (-1, BLOCK))
    most = y.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(min=-100))
    v = y / unit
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * unit).flatten(-2)


def _exact_cache(s):
    """Every slot's latent and rotated part, FP64."""
    L, R = s["case"]["latent"], s["case"]["rope"]
    c = s["latents"].reshape(-1, L).double()
    if s["scales"] is not None:
        c = c * torch.exp2(s["scales"].reshape(len(c), -1).double() - 127).repeat_interleave(BLOCK, 1)[:, :L]
    return c, s["ropes"].reshape(-1, R).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        at = case["dim"] - case["rotary"]
        x = s["x"].double()
        return torch.cat([x[..., :at], _exact_turn(x[..., at:], s, s["scale"])], -1)
    if case["op"] in ("write", "refill"):
        x = s["latent"].double()
        y = x * (x.square().mean(-1, keepdim=True) + NORM_EPS).rsqrt() * s["weight"].double()
        c, r = _exact_cache(s)
        r[s["slots"]] = _exact_turn(s["rope"].double()[:, None], s, 1.0)[:, 0]
        c[s["slots"]] = y if s["scales"] is None else _exact_codes(y)
        if case["op"] == "refill":
            return torch.cat([c[s["all_slots"]], r[s["all_slots"]]], -1)
        return c.view(s["latents"].shape), r.view(s["ropes"].shape)
    if case["op"] == "expanded":
        q, at, kv = s["q"].double(), s["query_start_loc"].tolist(), s["kv_start_loc"].tolist()
        out = torch.empty(case["tokens"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["new"]):
            r = s["k_rope"][kv[i]:kv[i + 1]].double()
            seen = torch.ones(n, s["lengths"][i], dtype=torch.bool, device="cuda").tril(s["lengths"][i] - n)
            for h in range(case["heads"]):
                k = torch.cat([s["k"][kv[i]:kv[i + 1], h].double(), r], 1)
                w = (q[at[i]:at[i + 1], h] @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                out[at[i]:at[i + 1], h] = torch.softmax(w, -1) @ s["v"][kv[i]:kv[i + 1], h].double()
        return out
    c, r = _exact_cache(s)
    out = torch.empty(s["q_latent"].shape, dtype=torch.float64, device="cuda")
    first, key = 0, 0
    for n, m in zip(s["new"], s["lengths"]):
        slots = s["all_slots"][key:key + m]
        k = c[slots]
        w = s["q_latent"][first:first + n].double() @ k.T + s["q_rope"][first:first + n].double() @ r[slots].T
        seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
        w = torch.softmax((w * s["scale"]).masked_fill(~seen[:, None], -math.inf), -1)
        out[first:first + n] = w @ k
        first, key = first + n, key + m
    return out
