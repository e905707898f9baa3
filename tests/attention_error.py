"""How far a row of attention may be from its FP64 definition: a bound on the row's norm that
grows with what the weights' roundings can do, not with the largest value of the cache, so that
a lost or doubled step of keys shows in long sequences too. Nothing here is the package's code."""

import torch

import latent_reference as ref


def rows(scores, seen, values):
    """(out, spread) of softmax(scores) @ values over the keys seen, FP64: spread is the root of
    sum_t p_t^2 |v_t|^2."""
    p = ref.softmax_rows(scores, seen)
    return p @ values, ((p * p) @ values.square().sum(-1, keepdim=True)).squeeze(-1).sqrt()


def bound(out, spread, dtype):
    """Of the error's norm, per row.

    A weight p_t rounded to `dtype` is off by d_t p_t, |d_t| <= h, half a step. The error is the
    vector sum_t d_t p_t v_t, of squared norm sum_t d_t^2 p_t^2 |v_t|^2, at most (h spread)^2, and
    terms of pairs of tokens. Roundings are independent and of mean 0, so these have mean 0 and,
    with v_t . v_s of size |v_t| |v_s| / sqrt(channels), a deviation of at most
    (h^2 / 3) sqrt(2 / channels) spread^2: with 32 channels or more, three of them are below
    (1 / 4) (h spread)^2, where one token does not hold all the weight; a factor 1.12 on the norm.
    Scores are FP32 sums of up to 576 products, each below 1 in size after scaling and turning into
    powers of two, so their own error is of size sqrt(576) 2^-24 times a few, below 2^-17: 2^-13 of
    a weight covers it, FP32 sums of the products and the hardware's exp2. The result rounds once,
    each channel by at most h of itself.
    """
    h = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return 1.12 * (h + 2.0 ** -13) * spread + h * out.norm(dim=-1) + tiny * out.shape[-1] ** 0.5


def worst(got, out, spread, dtype):
    """The largest error of a row, in bounds."""
    err = (got.double().cpu() - out).norm(dim=-1)
    return (err / bound(out, spread, dtype)).max().item()


def absorbed(q_latent, q_rope, cache, table, seq_lens, loc, scale):
    """(out, spread) of latent attention."""
    c, r = ref.values(*cache)
    pages, page = cache[0].shape[:2]
    out = torch.zeros(q_latent.shape, dtype=torch.float64)
    spread = torch.zeros(q_latent.shape[:2], dtype=torch.float64)
    for s in range(len(loc) - 1):
        a, b, n = int(loc[s]), int(loc[s + 1]), int(seq_lens[s])
        at = ref.slots_of(table[s], n, page, pages)
        k, kr = c[at], r[at]
        for i in range(a, b):
            seen = torch.arange(n) < n - (b - a) + (i - a) + 1
            w = (q_latent[i].double() @ k.T + q_rope[i].double() @ kr.T) * scale
            out[i], spread[i] = rows(w, seen.expand_as(w), k)
    return out, spread


def expanded(q, k, k_rope, v, loc, kv_loc, scale, causal=True):
    """(out, spread) of expanded attention."""
    out = torch.zeros(*q.shape[:2], v.shape[2], dtype=torch.float64)
    spread = torch.zeros(q.shape[:2], dtype=torch.float64)
    for s in range(len(loc) - 1):
        a, b, ka, kb = int(loc[s]), int(loc[s + 1]), int(kv_loc[s]), int(kv_loc[s + 1])
        n, m = b - a, kb - ka
        reach = torch.arange(n)[:, None] + (m - n) + 1 if causal else torch.full((n, 1), m)
        seen = torch.arange(m)[None] < reach
        for h in range(q.shape[1]):
            w = q[a:b, h, :k.shape[2]].double() @ k[ka:kb, h].double().T
            if k_rope is not None:
                w = w + q[a:b, h, k.shape[2]:].double() @ k_rope[ka:kb].double().T
            out[a:b, h], spread[a:b, h] = rows(w * scale, seen, v[ka:kb, h].double())
    return out, spread
