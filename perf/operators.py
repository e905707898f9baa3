"""Cases and plain forms of the gated delta rule and of the norms around it.

The cases stand for the part of a KDA layer that follows the packed short convolution:

- ``prefill``: the gated delta rule over packed sequences, read from the convolution's
  planes (3, tokens, heads * head_dim), with a paged FP32 state.
- ``decode``: its step for one token per sequence on the same state.
- ``gated``: the RMS norm per head after the rule, times its weight and an activated gate.
- ``residual``: the addition to the residual stream with a scale, and the norm before the
  next block.

``run`` computes a case's operator in its plain form where ``own`` is false, and makes the
package's calls where it is true. The plain forms work in FP32 (running sums of the log
decay in FP64), the prefill in chunks of up to 64 tokens. ``exact`` evaluates the
definitions in FP64, the delta rule one token after another.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
#: Row stride of the in_proj output (elements): the norm's gate and the decay gate are
#: column slices of such a projection.
PROJ = 9728
L2_EPS = 1e-6
NORM_EPS = 1e-5


# ---------------------------------------------------------------------------- cases


def _prefill(name, tokens, seqs, lengths, heads, qk_heads, dim, gate, dtype, initial):
    return {"name": name, "op": "prefill", "tokens": tokens, "seqs": seqs, "lengths": lengths,
            "heads": heads, "qk_heads": qk_heads, "dim": dim, "gate": gate, "dtype": dtype,
            "initial": initial}


def _decode(name, batch, heads, qk_heads, dim, gate, dtype):
    return {"name": name, "op": "decode", "batch": batch, "heads": heads, "qk_heads": qk_heads,
            "dim": dim, "gate": gate, "dtype": dtype}


def listed():
    return [
        # One short prompt on a rank with one head: latency counts.
        _prefill("prefill 64 tokens, 1 head", 64, 1, "equal", 1, 1, 128, "bounded", "bf16", 0.0),
        # A few short prompts scheduled together, 12 heads of 128 (3 x 1536 channels).
        _prefill("prefill 8 short prompts", 1204, 8, "uniform", 12, 12, 128, "softplus", "bf16", 0.5),
        # A whole prefill budget spent on one long prompt, continued from a stored state.
        _prefill("prefill 16384 tokens", 16384, 1, "equal", 12, 12, 128, "bounded", "bf16", 1.0),
        # The same budget over 64 prompts of very unequal lengths.
        _prefill("prefill 64 prompts", 16384, 64, "lognormal", 12, 12, 128, "bounded", "bf16", 0.75),
        # Many sequences of 1 to 4 tokens (speculative steps), 3 heads of 64: state traffic.
        _prefill("prefill 4096 x 1-4 tokens", 10240, 4096, "short", 3, 3, 64, "log", "bf16", 1.0),
        # An odd length in fp16, with every two value heads sharing a query and key head.
        _prefill("prefill 2999 tokens fp16", 2999, 3, "uniform", 8, 4, 128, "softplus", "f16", 0.5),
        # One token of one sequence: the step's latency.
        _decode("decode 1 sequence", 1, 12, 12, 128, "bounded", "bf16"),
        # An ordinary batch.
        _decode("decode 37 sequences", 37, 12, 12, 128, "softplus", "bf16"),
        # A full serving batch.
        _decode("decode 256 sequences", 256, 12, 12, 128, "bounded", "bf16"),
        # The norm after the rule: a decode batch, and a prefill budget.
        {"name": "gated norm 37 tokens", "op": "gated", "tokens": 37, "heads": 12, "dim": 128,
         "activation": "sigmoid", "dtype": "bf16"},
        {"name": "gated norm 16384 tokens", "op": "gated", "tokens": 16384, "heads": 12, "dim": 128,
         "activation": "sigmoid", "dtype": "bf16"},
        # The residual addition and the norm before a block, over a prefill budget.
        {"name": "residual norm 16384 tokens", "op": "residual", "tokens": 16384, "hidden": 4096,
         "scale": 0.25, "dtype": "bf16"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "gated", "residual"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("prefill", "decode"):
        dim = rng.choice([64, 128])
        qk = rng.choice([1, 2, 3, 4, 6, 8, 12])
        heads = qk * rng.choice([1, 1, 2]) if qk <= 6 else qk
        gate = rng.choice(["bounded", "softplus", "log"])
        if op == "decode":
            most = min(512, 256 * 12 * 128 * 128 // (heads * dim * dim))
            return {"op": op, "batch": _log_int(rng, 1, most), "heads": heads, "qk_heads": qk,
                    "dim": dim, "gate": gate, "dtype": dtype}
        tokens = _log_int(rng, 1, min(16384, 16384 * 1536 // (heads * dim)))
        # A sequence costs its state, read and written, beside its tokens.
        seqs = _log_int(rng, 1, max(1, min(tokens, 512)))
        return {"op": op, "tokens": tokens, "seqs": seqs,
                "lengths": rng.choice(["equal", "uniform", "lognormal"]), "heads": heads,
                "qk_heads": qk, "dim": dim, "gate": gate, "dtype": dtype,
                "initial": rng.choice([0.0, 0.5, 1.0])}
    if op == "gated":
        return {"op": op, "tokens": _log_int(rng, 1, 16384 if dtype != "f32" else 8192),
                "heads": rng.randint(1, 12), "dim": rng.choice([64, 128]),
                "activation": rng.choice(["sigmoid", "silu"]), "dtype": dtype}
    hidden = 40 * _log_int(rng, 13, 204) + rng.choice([0, 0, 0, 1])
    most = min(16384, 16384 * 4096 // hidden) // (2 if dtype == "f32" else 1)
    return {"op": op, "tokens": _log_int(rng, 1, most), "hidden": hidden,
            "scale": rng.choice([1.0, 0.25, 0.7]), "dtype": dtype}


# --------------------------------------------------------------------------- inputs


def _lengths(case, seed):
    """Token counts of the case's sequences (host integers), summing to its tokens."""
    tokens, seqs, kind = case["tokens"], case["seqs"], case["lengths"]
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    if kind == "equal":
        return [tokens // seqs + (i < tokens % seqs) for i in range(seqs)]
    if kind == "short":
        # 1 to 4 each: start from 1 and hand out the rest.
        n = torch.randint(1, 5, (seqs,), generator=g)
        order = torch.randperm(seqs, generator=g)
        excess = int(n.sum()) - tokens
        step = -1 if excess > 0 else 1
        room = torch.where(n[order] + step >= 1, n[order] + step <= 4, False)
        change = order[room.nonzero().flatten()[: abs(excess)]]
        n[change] += step
        n[-1] += tokens - int(n.sum())  # what is left, if anything
        return [int(x) for x in n]
    if kind == "uniform":
        w = torch.rand(seqs, generator=g, dtype=torch.float64) + 0.02
    else:
        w = torch.exp(torch.randn(seqs, generator=g, dtype=torch.float64))
    ends = torch.round(torch.cumsum(w, 0) / w.sum() * tokens).to(torch.int64)
    ends[-1] = tokens
    return [int(x) for x in torch.diff(ends, prepend=torch.zeros(1, dtype=torch.int64))]


def _rule_inputs(case, seed, tokens, seqs, initial):
    """Tensors that both forms of the delta rule take."""
    dev, dt = "cuda", DTYPES[case["dtype"]]
    H, HK, D = case["heads"], case["qk_heads"], case["dim"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, device=dev) * scale + shift

    # q, k and v come out of the convolution's SiLU, as planes.
    x = normal(tokens, (2 * HK + H) * D)
    x = (x * torch.sigmoid(x)).to(dt)
    q = x[:, : HK * D].contiguous().view(tokens, HK, D)
    k = x[:, HK * D: 2 * HK * D].contiguous().view(tokens, HK, D)
    v = x[:, 2 * HK * D:].contiguous().view(tokens, H, D)
    s = {"case": case, "q": q, "k": k, "v": v}
    # The decay gate: columns of a projection's rows, or a ready log decay in FP32.
    if case["gate"] == "log":
        s["g"] = -torch.exp(normal(tokens, H, D, scale=1.0, shift=-3.0))
        s["a_log"] = s["dt_bias"] = s["lower_bound"] = None
    else:
        rows = normal(tokens, max(H * D + 64, PROJ // 4)).to(dt)
        s["g"] = rows[:, 32: 32 + H * D].view(tokens, H, D)
        s["a_log"] = torch.log(torch.rand(H, generator=g, device=dev) * 15 + 1)
        if case["gate"] == "softplus":
            # softplus(dt_bias) log-uniform in [0.001, 0.1], as such layers start out
            u = torch.rand(H, D, generator=g, device=dev) * math.log(100.0) + math.log(0.001)
            s["dt_bias"] = torch.log(torch.expm1(torch.exp(u)))
            s["lower_bound"] = None
        else:
            s["a_log"] = s["a_log"] * 0.25
            s["dt_bias"] = normal(H, D, scale=1.0, shift=-2.0)
            s["lower_bound"] = -5.0
    s["beta"] = normal(tokens, H).to(dt)  # logits; beta = sigmoid
    lines = seqs + 3
    s["states"] = normal(lines, H, D, D, scale=0.3)
    s["lines"] = torch.randperm(lines, generator=g, device=dev)[:seqs].to(torch.int32)
    s["initial"] = torch.rand(seqs, generator=g, device=dev) < initial
    return s


def prepare(case, seed):
    dev = "cuda"
    if case["op"] == "prefill":
        lengths = _lengths(case, seed)
        s = _rule_inputs(case, seed, case["tokens"], case["seqs"], case["initial"])
        starts = [0]
        for n in lengths:
            starts.append(starts[-1] + n)
        s["query_start_loc"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["lengths"] = lengths
        s["plan"] = _chunk_plan(lengths, starts, dev)
        return s
    if case["op"] == "decode":
        return _rule_inputs(case, seed, case["batch"], case["batch"], 1.0)
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "gated":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        x = (torch.randn(T, H, D, generator=g, device=dev) * 0.3).to(dt)
        rows = torch.randn(T, H * D + 64, generator=g, device=dev).to(dt)
        w = 1 + 0.1 * torch.randn(D, generator=g, device=dev)
        return {"case": case, "x": x, "gate": rows[:, 64:].view(T, H, D), "weight": w}
    T, N = case["tokens"], case["hidden"]
    return {"case": case, "x": torch.randn(T, N, generator=g, device=dev).to(dt),
            "residual": (2 * torch.randn(T, N, generator=g, device=dev)).to(dt),
            "weight": 1 + 0.1 * torch.randn(N, generator=g, device=dev)}


def _chunk_plan(lengths, starts, dev):
    """Where the plain prefill's chunks lie, from the lengths alone: the token of each
    chunk row (the row after the last token stands for padding) and, for each step, the
    sequences that still have a chunk and which chunk that is."""
    longest = max(lengths)
    size = min(64, max(1, longest))
    tokens = starts[-1]
    n = torch.tensor(lengths, dtype=torch.int64)
    per = (n + size - 1) // size
    first = torch.cumsum(per, 0) - per
    seq = torch.repeat_interleave(torch.arange(len(lengths)), per)
    j = torch.arange(len(seq)) - first[seq]
    row = j[:, None] * size + torch.arange(size)[None]
    at = torch.where(row < n[seq][:, None], row + torch.tensor(starts)[:-1][seq][:, None], tokens)
    steps = []
    for i in range(int(per.max())):
        s = (per > i).nonzero().flatten()
        steps.append((s.to(dev), (first[s] + i).to(dev)))
    return {"size": size, "rows": at.to(dev), "steps": steps}


# ---------------------------------------------------------------------- plain forms


def _log_decay(s, dtype):
    """Log decay of every token, head and channel."""
    g = s["g"].to(dtype)
    if s["a_log"] is None:
        return g
    a = torch.exp(s["a_log"].to(dtype))[:, None]
    x = g + s["dt_bias"].to(dtype)
    if s["lower_bound"] is not None:
        return s["lower_bound"] / (1 + torch.exp(-a * x))
    return -a * (torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x))))


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + L2_EPS)


def _plain_prefill(s):
    case, plan = s["case"], s["plan"]
    T, H, D = case["tokens"], case["heads"], case["dim"]
    share = H // case["qk_heads"]
    C, rows = plan["size"], plan["rows"]

    def chunks(x):
        """(tokens, H, ...) as (chunks, H, C, ...), zeros where a chunk has no token."""
        x = torch.cat([x, torch.zeros_like(x[:1])])[rows]
        return x.transpose(1, 2)

    q = chunks(_unit(s["q"].float()).repeat_interleave(share, 1) * D ** -0.5)
    k = chunks(_unit(s["k"].float()).repeat_interleave(share, 1))
    v = chunks(s["v"].float())
    beta = chunks(torch.sigmoid(s["beta"].float()))[..., None]
    G = torch.cumsum(chunks(_log_decay(s, torch.float64)), 2)
    below = torch.tril(torch.ones(C, C, dtype=torch.bool, device=rows.device))[:, :, None]
    W = (G[:, :, :, None] - G[:, :, None]).float()
    W = torch.exp(torch.where(below, W, -math.inf)) * k[:, :, None]  # decay from i to t, times k_i
    Akk = (W * k[:, :, :, None]).sum(-1)
    Aqk = (W * q[:, :, :, None]).sum(-1)
    del W
    L = torch.tril(Akk, -1) * beta
    decayed = torch.exp(G).float()
    last = G[:, :, -1:]
    kend = (k * torch.exp(last - G).float()).transpose(2, 3)
    qg = q * decayed
    # X = (I + L)^-1 beta [v, k e^G], row by row
    X = torch.cat([v, k * decayed], -1) * beta
    for t in range(1, C):
        X[:, :, t] -= (L[:, :, t:t + 1, :t] @ X[:, :, :t])[:, :, 0]
    Xv, Xk = X[..., :D], X[..., D:]
    end = torch.exp(last).float().transpose(2, 3)
    lines = s["lines"].long()
    S = s["states"][lines] * s["initial"][:, None, None, None]
    o = torch.empty(len(rows), H, C, D, device=rows.device)
    for seqs, at in plan["steps"]:
        S0 = S[seqs]
        U = Xv[at] - Xk[at] @ S0
        o[at] = qg[at] @ S0 + Aqk[at] @ U
        S[seqs] = S0 * end[at] + kend[at] @ U
    s["states"][lines] = S
    out = torch.empty(T + 1, H, D, dtype=s["v"].dtype, device=rows.device)
    out[rows] = o.transpose(1, 2).to(out.dtype)
    return out[:T], s["states"]


def _plain_decode(s):
    share = s["case"]["heads"] // s["case"]["qk_heads"]
    D = s["case"]["dim"]
    q = _unit(s["q"].float()).repeat_interleave(share, 1) * D ** -0.5
    k = _unit(s["k"].float()).repeat_interleave(share, 1)
    beta = torch.sigmoid(s["beta"].float())[..., None]
    lines = s["lines"].long()
    S = s["states"][lines] * torch.exp(_log_decay(s, torch.float32))[..., None]
    u = (s["v"].float() - (S * k[..., None]).sum(-2)) * beta
    S = S + k[..., None] * u[..., None, :]
    s["states"][lines] = S
    return (S * q[..., None]).sum(-2).to(s["v"].dtype), s["states"]


def _plain_gated(s):
    x, z = s["x"].float(), s["gate"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * s["weight"]
    y = y * torch.sigmoid(z)
    if s["case"]["activation"] == "silu":
        y = y * z
    return y.to(s["x"].dtype)


def _plain_residual(s):
    h = s["residual"].float() + s["case"]["scale"] * s["x"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + NORM_EPS) * s["weight"]
    s["residual"].copy_(h)
    return y.to(s["x"].dtype), s["residual"]


# ------------------------------------------------------------------- the package's calls


def _own(s):
    import packed_varlen_causal_depthwise_amd as kd

    case = s["case"]
    if case["op"] == "prefill":
        out = kd.gated_delta_rule_fn(
            s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["query_start_loc"],
            s["lines"], s["initial"], a_log=s["a_log"], dt_bias=s["dt_bias"],
            lower_bound=s["lower_bound"], beta_logits=True, null_block_id=None)
        return out, s["states"]
    if case["op"] == "decode":
        out = kd.gated_delta_rule_update(
            s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["lines"],
            a_log=s["a_log"], dt_bias=s["dt_bias"], lower_bound=s["lower_bound"],
            beta_logits=True, null_block_id=None)
        return out, s["states"]
    if case["op"] == "gated":
        return kd.gated_rms_norm(s["x"], s["gate"], s["weight"], eps=NORM_EPS,
                                 activation=case["activation"])
    out = kd.residual_rms_norm(s["x"], s["residual"], s["weight"], eps=NORM_EPS,
                               residual_scale=case["scale"])
    return out, s["residual"]


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "gated": _plain_gated,
            "residual": _plain_residual}[state["case"]["op"]](state)


# ------------------------------------------------------------------------ work and truth


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("prefill", "decode"):
        H, HK, D = case["heads"], case["qk_heads"], case["dim"]
        tokens = case["tokens"] if case["op"] == "prefill" else case["batch"]
        seqs = case["seqs"] if case["op"] == "prefill" else case["batch"]
        initial = case["initial"] if case["op"] == "prefill" else 1.0
        gate = 4 if case["gate"] == "log" else e
        b = tokens * D * (e * (2 * HK + 2 * H) + gate * H) + tokens * H * e
        b += int(4 * D * D * H * seqs * (1 + initial)) + 9 * seqs
        # decay, key product, update and query product of a token's state
        return {"bytes": b, "flops": 7 * D * D * H * tokens}
    if case["op"] == "gated":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 3 * e * n + 4 * case["dim"], "flops": 10 * n}
    n = case["tokens"] * case["hidden"]
    return {"bytes": 4 * e * n + 4 * case["hidden"], "flops": 6 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated":
        x, z = s["x"].double(), s["gate"].double()
        y = x / (x.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * s["weight"].double()
        y = y / (1 + torch.exp(-z))
        return y * z if case["activation"] == "silu" else y
    if case["op"] == "residual":
        h = s["residual"].double() + case["scale"] * s["x"].double()
        y = h / (h.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * s["weight"].double()
        return y, h
    share = case["heads"] // case["qk_heads"]
    q, k = s["q"].double(), s["k"].double()
    q = (q / (q.square().sum(-1, keepdim=True) + L2_EPS).sqrt()).repeat_interleave(share, 1)
    k = (k / (k.square().sum(-1, keepdim=True) + L2_EPS).sqrt()).repeat_interleave(share, 1)
    q = q / math.sqrt(case["dim"])
    v, beta = s["v"].double(), 1 / (1 + torch.exp(-s["beta"].double()))
    decay = torch.exp(_log_decay(s, torch.float64))
    lengths = s["lengths"] if case["op"] == "prefill" else [1] * case["batch"]
    first = [0]
    for n in lengths:
        first.append(first[-1] + n)
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])  # longest first
    pick = torch.tensor(order, device="cuda")
    start = torch.tensor(first[:-1], device="cuda")[pick]
    S = s["states"].double()[s["lines"].long()[pick]] * s["initial"][pick][:, None, None, None]
    if case["op"] == "decode":
        S = s["states"].double()[s["lines"].long()[pick]]
    o = torch.zeros_like(v)
    live = len(order)
    for t in range(max(lengths)):
        while lengths[order[live - 1]] <= t:
            live -= 1
        at = start[:live] + t
        A = S[:live]
        A *= decay[at][..., None]
        kt = k[at]
        u = beta[at][..., None] * (v[at] - torch.einsum("nhk,nhkv->nhv", kt, A))
        A += kt[..., None] * u[:, :, None]
        o[at] = torch.einsum("nhk,nhkv->nhv", q[at], A)
    states = s["states"].double()
    states[s["lines"].long()[pick]] = S
    return o, states
