"""Absorbed latent attention: values that are not finite reach the rows that see them, no others."""

import pytest
import torch

import attention_error as ae
import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
INF = float("inf")


def normal(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def inputs(new, lens, heads, dtype, e4m3=False, latent=256, rope=64, page=16):
    """(q_latent, q_rope, (latents, ropes, scales), table, seq_lens, loc) on the CPU."""
    table, pages = ref.tables(lens, page)
    cache = ref.cache(pages, page, latent, rope, dtype, e4m3)
    q, r = normal(sum(new), heads, latent, seed=1, dtype=dtype), normal(sum(new), heads, rope, seed=2, dtype=dtype)
    return q, r, cache, table, torch.tensor(lens, dtype=torch.int32), ref.starts(new)


def run(q, r, cache, table, lens, loc):
    return kd.latent_attention_fn(*ref.on_gpu(q, r, *cache, table, lens, loc), scale=0.1).cpu()


def put(latents, slot, channel, value):
    """A copy of the latents with one slot's channel changed (NaN alone in 8 bits)."""
    latents = latents.clone()
    if latents.dtype == torch.float8_e4m3fn:
        latents.view(torch.uint8).flatten(0, 1)[slot, channel] = 0x7F
    else:
        latents.flatten(0, 1)[slot, channel] = value
    return latents


@DTYPES
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("value", [float("nan"), INF])
@pytest.mark.parametrize("new,lens,heads", [
    # A block's rows (16, 32 or 64 by the average) are one token's: heads fill it ...
    ([2], [40], 64), ([3], [3000], 128), ([2, 5], [33, 70], 64), ([4], [4], 192),
    # ... or sequences without new tokens lower the average.
    ([2, 0], [40, 9], 16), ([2, 0], [40, 0], 32), ([2, 0, 0, 0], [600, 1, 0, 3], 32), ([4, 0, 0, 0, 1], [77, 0, 0, 5, 64], 16),
    # Blocks of several tokens, and parts of them.
    ([5], [40], 16), ([6, 1], [40, 64], 3), ([3], [70], 40), ([7], [2000], 12)])
def test_later_tokens(new, lens, heads, value, e4m3, dtype):
    """The last token of the first sequence, and a new one before it, where there is one."""
    if e4m3 and value == INF:
        pytest.skip("8-bit latents have no infinity")
    q, r, cache, table, seq_lens, loc = inputs(new, lens, heads, dtype, e4m3)
    clean = run(q, r, cache, table, seq_lens, loc)
    assert torch.isfinite(clean).all()
    want, spread = ae.absorbed(q, r, cache, table, seq_lens, loc, 0.1)
    at = ref.slots_of(table[0], lens[0], 16, cache[0].shape[0])
    for token in sorted({new[0] - 1, (new[0] + 1) // 2}):  # of the new ones
        bad = put(cache[0], at[lens[0] - new[0] + token], 5, value)
        got = run(q, r, (bad, *cache[1:]), table, seq_lens, loc)
        assert torch.equal(got[new[0]:], clean[new[0]:]), "reaches another sequence"
        if value == INF and token > 0:
            # A score of inf is a row's new largest, and then the sums of all rows of its wave are
            # rescaled: weights of the others are rounded at another power, still by half a step.
            assert ae.worst(got[:token], want[:token], spread[:token], dtype) < 1, "reaches an earlier token"
        else:
            assert torch.equal(got[:token], clean[:token]), "reaches an earlier token"
        assert not torch.isfinite(got[token:new[0], :, 5]).any()
        # (The score of a NaN is NaN; that of an infinity an infinity of either sign.)
        assert value == INF or torch.isnan(got[token:new[0]]).all()


@DTYPES
@pytest.mark.parametrize("new,lens,heads", [
    ([6], [40], 3), ([6, 1], [70, 64], 12), ([5], [40], 16), ([3], [70], 40), ([2], [40], 64), ([7], [4000], 12),
    ([30, 2], [3000, 500], 8), ([2, 0], [40, 9], 16)])
@pytest.mark.parametrize("kind", ["inf", "-inf", "8 bits"])
def test_weightless_infinities(new, lens, heads, kind, dtype):
    """A token whose infinite latent gives it a score of -inf has weight 0: 0 times an infinity
    is NaN in that channel, whatever other rows see, and nothing in the others."""
    if kind == "8 bits" and dtype != F16:
        pytest.skip("values past fp16's range")
    q, r, cache, table, seq_lens, loc = inputs(new, lens, heads, dtype, kind == "8 bits")
    q[..., 5] = 1.0 if kind == "-inf" else -1.0
    at = ref.slots_of(table[0], lens[0], 16, cache[0].shape[0])
    for key in sorted({0, lens[0] // 2, lens[0] - new[0], lens[0] - new[0] // 2 - 1}):
        slot = at[key]
        outs = []
        # What weighs nothing either: -30000 * 0.1.
        for value in (float(kind), -30000.0 if kind == "-inf" else 30000.0) if kind != "8 bits" else (448, 224):
            latents, scales = cache[0].clone(), cache[2]
            if kind == "8 bits":  # 448 * 2^8 is past fp16's end, 224 * 2^8 before it
                scales = scales.clone()
                scales.flatten(0, 1)[slot, 0] = 135
                codes = torch.zeros(32)
                codes[5] = value
                latents.view(torch.uint8).flatten(0, 1)[slot, :32] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                latents.flatten(0, 1)[slot, 5] = value
            outs.append(run(q, r, (latents, cache[1], scales), table, seq_lens, loc))
        got, want = outs
        assert torch.isfinite(want).all()
        first = max(0, key - (lens[0] - new[0]))  # the first row that sees it
        assert torch.isnan(got[first:new[0], :, 5]).all(), key
        got[first:new[0], :, 5] = want[first:new[0], :, 5]
        assert torch.equal(got, want), key
