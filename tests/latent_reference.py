"""Latent attention, its cache and its rotation from their definitions in FP64 on the CPU, and
the inputs that their tests share. Nothing here is the package's code."""

import math

import torch

BLOCK = 32


def frequencies(rotary, base=10000.0):
    return (base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).float()


def turned(x, positions, inv_freq, interleaved, scale=1.0):
    """x (tokens, heads, rotary), every pair turned, FP64."""
    x, a = x.double(), positions.double()[:, None, None] * inv_freq.double()
    c, s = scale * torch.cos(a), scale * torch.sin(a)
    out = torch.empty_like(x)
    half = x.shape[-1] // 2
    first = slice(0, None, 2) if interleaved else slice(0, half)
    second = slice(1, None, 2) if interleaved else slice(half, None)
    u, v = x[..., first], x[..., second]
    out[..., first] = u * c - v * s
    out[..., second] = u * s + v * c
    return out


def normed(x, weight, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.double()


def to_8_bits(y):
    """(values in units, scale bytes) of y (..., latent), rounded to FP32 first: per block of 32
    the smallest e >= -100 with every finite |y| <= 448 * 2^e, then 4 significant bits, to
    nearest even, in steps of 2^-9 and more."""
    y = y.float().double().unflatten(-1, (-1, BLOCK))
    finite = torch.isfinite(y)
    most = torch.where(finite, y.abs(), 0.0).amax(-1, keepdim=True)
    e = torch.full_like(most, -100.0)
    for _ in range(300):
        e = torch.where(most > 448 * torch.exp2(e), e + 1, e)
    v = torch.where(finite, y, 0.0) * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    v = torch.where(finite, torch.round(v / step) * step, float("nan"))
    return v.flatten(-2), (e + 127).squeeze(-1).to(torch.uint8)


def values(latents, ropes, scales):
    """Every slot's (latent, rotated part), FP64."""
    c = latents.double().flatten(0, 1)
    if scales is not None:
        s = torch.exp2(scales.double().flatten(0, 1) - 127)
        c = c * s.repeat_interleave(BLOCK, -1)
    return c, ropes.double().flatten(0, 1)


def slots_of(table, length, page, pages):
    """The slots of a sequence's tokens; -1 where its page is outside the cache."""
    i = torch.arange(length)
    ok = i // page < table.shape[0]
    at = table[(i // page).clamp(max=max(0, table.shape[0] - 1))].long() if table.shape[0] else i
    ok &= (at >= 0) & (at < pages)
    return torch.where(ok, at * page + i % page, -1)


def softmax_rows(w, seen):
    """Softmax of each row over the keys it sees, zeros for a row without any."""
    w = w.masked_fill(~seen, -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-1e300) if w.shape[-1] else w
    p = torch.where(seen, torch.exp(w - top), 0.0)
    z = p.sum(-1, keepdim=True)
    return torch.where(z > 0, p / z.clamp(min=1e-300), 0.0)


def attention(q_latent, q_rope, latents, ropes, scales, table, seq_lens, loc, scale):
    """Absorbed attention, FP64; rows no sequence owns are NaN."""
    c, r = values(latents, ropes, scales)
    pages, page = latents.shape[:2]
    out = torch.full(q_latent.shape, float("nan"), dtype=torch.float64)
    for s in range(len(loc) - 1):
        a, b = int(loc[s]), int(loc[s + 1])
        n = int(seq_lens[s])
        at = slots_of(table[s], max(0, min(n, table.shape[1] * page)), page, pages)
        k, kr = c[at.clamp(min=0)], r[at.clamp(min=0)]
        for i in range(a, b):
            seen = (at >= 0) & (torch.arange(len(at)) < n - (b - a) + (i - a) + 1)
            w = (q_latent[i].double() @ k.T + q_rope[i].double() @ kr.T) * scale
            p = softmax_rows(w.masked_fill(~seen, 0.0), seen.expand_as(w))
            out[i] = p @ torch.where(seen[:, None], k, 0.0)
    return out


def expanded(q, k, k_rope, v, loc, kv_loc, scale, causal=True):
    """Expanded attention, FP64; rows no sequence owns are NaN."""
    H, D = q.shape[1], k.shape[2]
    out = torch.full((q.shape[0], H, v.shape[2]), float("nan"), dtype=torch.float64)
    for s in range(len(loc) - 1):
        a, b, ka, kb = int(loc[s]), int(loc[s + 1]), int(kv_loc[s]), int(kv_loc[s + 1])
        n, m = b - a, kb - ka
        reach = torch.arange(n)[:, None] + (m - n) + 1 if causal else torch.full((n, 1), m)
        seen = torch.arange(m)[None] < reach
        for h in range(H):
            w = q[a:b, h, :D].double() @ k[ka:kb, h].double().T
            if k_rope is not None:
                w = w + q[a:b, h, D:].double() @ k_rope[ka:kb].double().T
            out[a:b, h] = softmax_rows(w * scale, seen) @ v[ka:kb, h].double()
    return out


def cache(pages, page, latent, rope, dtype, e4m3=False, seed=0, one_tensor=False):
    """A cache of random tokens (latents, ropes, scales or None), CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    if one_tensor:
        both = torch.randn(pages, page, latent + rope, generator=g).to(dtype)
        return both[..., :latent], both[..., latent:], None
    ropes = torch.randn(pages, page, rope, generator=g).to(dtype)
    if not e4m3:
        return torch.randn(pages, page, latent, generator=g).to(dtype), ropes, None
    codes = (torch.randn(pages, page, latent, generator=g) * 100).clamp(-448, 448)
    scales = torch.randint(118, 122, (pages, page, latent // BLOCK), generator=g)
    return codes.to(torch.float8_e4m3fn), ropes, scales.to(torch.uint8)


def tables(lengths, page, seed=0, spare=2, width=None):
    """Pages at random places for sequences of these lengths: (table, number of pages); entries
    past a sequence's pages lie far outside any cache."""
    per = [(n + page - 1) // page for n in lengths]
    pages = sum(per) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lengths), max(per + [1]) if width is None else width), 1 << 30, dtype=torch.int32)
    first = 0
    for s, n in enumerate(per):
        table[s, :n] = order[first:first + n]
        first += n
    return table, pages


def starts(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)


def on_gpu(*tensors):
    """The same tensors on the GPU, strides kept (slices of one tensor become separate ones)."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        shape = [(n - 1) * s for n, s in zip(t.shape, t.stride())]
        flat = t.as_strided((sum(shape) + 1 if t.numel() else 0,), (1,))
        out.append(flat.cuda().as_strided(t.shape, t.stride()) if t.numel() else t.cuda())
    return out
