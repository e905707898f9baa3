"""Plain FP64 forms of the gated delta rule and the norms, and inputs for their tests.

The rule is evaluated one token after another, straight from its definition
(include/kdaconv.h). Tensors are on the CPU.

Tolerances. An output is rounded once, by at most half a step: eps(dtype) / 2 of its value.
Before that the arithmetic holds FP32 (2^-24 per operation) or pairs of 22 bits; a value
passes through about 8 products and through sums whose rounding errors add up like a
random walk, and exp of a log decay of size G carries 2^-24 G (contributions with G over
16 are below 2^-23 themselves). 2^-17 of the norm, or of the largest value for single
elements, leaves a factor of about 8 over 2^-22 * 4 for that. Both bounds were set before
the first run.
"""

from __future__ import annotations

import torch

ARITHMETIC = 2.0 ** -17
L2_EPS = 1e-6


def log_decay(g, a_log, dt_bias, lower_bound):
    g = g.double()
    if a_log is None:
        return g
    a = torch.exp(a_log.double())[:, None]
    x = g if dt_bias is None else g + dt_bias.double().view(1, *g.shape[1:])
    if lower_bound is None:
        return -a * torch.nn.functional.softplus(x, threshold=700.0)
    return lower_bound * torch.sigmoid(a * x)


def delta_rule(q, k, v, g, beta, states, query_start_loc, cache_indices, has_initial_state, *,
               a_log=None, dt_bias=None, lower_bound=None, beta_logits=False, qk_l2norm=True,
               scale=None, null_block_id=None):
    """(out float64 with NaN in rows no sequence owns, states float64 after the call)."""
    tokens, heads, dim = v.shape
    share = heads // q.shape[1]
    q = q.double().repeat_interleave(share, 1)
    k = k.double().repeat_interleave(share, 1)
    v = v.double()
    if g.dim() == 2:
        g = g[..., None].expand(tokens, heads, dim)
    if qk_l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + L2_EPS).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + L2_EPS).sqrt()
    q = q * (dim ** -0.5 if scale is None else scale)
    b = torch.sigmoid(beta.double()) if beta_logits else beta.double()
    decay = torch.exp(log_decay(g, a_log, dt_bias, lower_bound))
    out = torch.full((tokens, heads, dim), float("nan"), dtype=torch.float64)
    states = states.double().clone()
    loc = query_start_loc.tolist()
    for s in range(len(loc) - 1):
        line = int(cache_indices[s])
        stored = 0 <= line < len(states) and line != null_block_id
        start = stored and has_initial_state is not None and bool(has_initial_state[s])
        S = states[line].clone() if start else torch.zeros(heads, dim, dim, dtype=torch.float64)
        for t in range(loc[s], loc[s + 1]):
            S = S * decay[t][..., None]
            u = b[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
            S = S + k[t][..., None] * u[:, None]
            out[t] = torch.einsum("hk,hkv->hv", q[t], S)
        if stored:
            states[line] = S
    return out, states


def gated_norm(x, gate, weight, eps, activation):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    if gate is not None:
        z = gate.double()
        y = y * torch.sigmoid(z) * (z if activation == "silu" else 1.0)
    return y


def residual_norm(x, residual, weight, eps, scale):
    h = x.double() * scale + (0.0 if residual is None else residual.double())
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return (y if weight is None else y * weight.double()), h


def rule_inputs(lengths, heads=2, qk_heads=None, dim=128, dtype=torch.bfloat16, *, seed=0,
                gate="bounded", gate_dtype=None, per_head=False, beta_dtype=None, logits=True,
                lines=None, pad=0, strided=False, initial=None, v_scale=1.0, state_scale=0.3):
    """CPU tensors and keyword arguments of one call."""
    qk_heads = heads if qk_heads is None else qk_heads
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    S, T = len(lengths), sum(lengths) + pad
    x = normal(T, (2 * qk_heads + heads) * dim)
    x = x * torch.sigmoid(x)
    x[:, 2 * qk_heads * dim:] *= v_scale
    x = x.to(dtype)
    if strided:  # columns of wider rows, starting at an odd column
        wide = torch.full((T, x.shape[1] + 37), float("nan"), dtype=dtype)
        wide[:, 3: 3 + x.shape[1]] = x
        x = wide[:, 3: 3 + x.shape[1]]
    a, b = qk_heads * dim, 2 * qk_heads * dim
    q, k, v = (x[:, :a].unflatten(1, (qk_heads, dim)), x[:, a:b].unflatten(1, (qk_heads, dim)),
               x[:, b:].unflatten(1, (heads, dim)))
    gd = dtype if gate_dtype is None else gate_dtype
    kw = dict(beta_logits=logits)
    shape = (T, heads) if per_head else (T, heads, dim)
    if gate == "log":
        g = (-torch.exp(normal(*shape) - 3.0)).to(gd)
    else:
        g = normal(*shape).to(gd)
        kw["a_log"] = torch.rand(heads, generator=gen) * 2.0
        kw["dt_bias"] = normal(heads, dim) - 3.0
        kw["lower_bound"] = -5.0 if gate == "bounded" else None
    beta = normal(T, heads) if logits else torch.rand(T, heads, generator=gen)
    beta = beta.to(dtype if beta_dtype is None else beta_dtype)
    lines = S + 2 if lines is None else lines
    states = normal(lines, heads, dim, dim) * state_scale * v_scale
    ci = torch.randperm(lines, generator=gen)[:S].to(torch.int32)
    if initial is None:
        initial = torch.rand(S, generator=gen) < 0.5
    loc = torch.zeros(S + 1, dtype=torch.int32)
    loc[1:] = torch.tensor(lengths, dtype=torch.int32).cumsum(0)
    return [q, k, v, g, beta, states, loc, ci, initial], kw


def check(got, want, dtype, what):
    """got against the FP64 want: every element, and the whole."""
    assert got.shape == want.shape
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    half = torch.finfo(dtype).eps / 2
    err = (got - want).abs()
    top = want.abs().max()
    # FP16 and FP32 subnormal steps: half of the smallest
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    bound = half * want.abs() + ARITHMETIC * top + tiny
    bad = (err > bound).sum().item()
    assert bad == 0, f"{what}: {bad} of {err.numel()} elements off, worst {(err / bound).max():.3g} of the bound"
    norm = want.norm()
    if norm > 0:
        rel = ((got - want).norm() / norm).item()
        # a rounding to `dtype` is off by half a step at most: its norm is, too
        assert rel <= half + ARITHMETIC + tiny * err.numel() ** 0.5 / norm, f"{what}: norm {rel:.3g}"
