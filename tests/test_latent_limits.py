"""Limits of the latent attention operators on the host: what is refused, and what is not."""

import math

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from packed_varlen_causal_depthwise_amd._lib import EINVAL, EUNSUPPORTED, OK
from test_latent_boundary import A, expanded_code, rotary_code, write_code

FAR = 1 << 40


@pytest.mark.parametrize("kw,code", [
    # Heads may be as far apart as they are, and so may queries.
    (dict(q0=192, q1=FAR), OK), (dict(q0=FAR + 1, q1=192), OK), (dict(k0=128, k1=1 << 23), OK), (dict(k0=128, k1=FAR), OK),
    (dict(v0=128, v1=FAR), OK), (dict(q1=1 << 23, k1=1 << 23, v1=1 << 23), OK),
    (dict(k1=FAR + 4), EUNSUPPORTED), (dict(v1=FAR + 7), EUNSUPPORTED), (dict(q1=-1), EUNSUPPORTED), (dict(v1=-8), EUNSUPPORTED),
    # Tokens of keys and values are counted in 32 bits from a step's first.
    (dict(k0=(1 << 23) - 8), OK), (dict(kr0=(1 << 23) - 8), OK), (dict(v0=(1 << 23) - 8), OK),
    (dict(k0=1 << 23), EUNSUPPORTED), (dict(kr0=1 << 23), EUNSUPPORTED), (dict(v0=FAR), EUNSUPPORTED),
    (dict(k0=FAR, v0=FAR, kr0=FAR, keys=1), OK), (dict(kr0=FAR, rope=0), OK), (dict(k1=FAR + 1, heads=1), OK),
])
def test_expanded_strides(kw, code):
    assert expanded_code(**kw) == code


def test_supported_allocates_nothing(monkeypatch):
    """Queries of support look at the tensors alone."""
    bf = torch.bfloat16
    cache = ref.cache(4, 8, 64, 16, bf)
    q, r = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 2, 16, dtype=bf)
    k, v, kr = torch.zeros(9, 2, 64, dtype=bf), torch.zeros(9, 2, 64, dtype=bf), torch.zeros(9, 16, dtype=bf)
    long = torch.cat((q, r), -1)
    for name in ("empty", "zeros", "ones", "full", "empty_like", "tensor"):
        monkeypatch.setattr(torch, name, None)
    assert not kd.latent_attention_supported(q, r, *cache)  # not on a GPU
    assert not kd.latent_attention_supported(q, r[:, :1], *cache)
    assert not kd.expanded_attention_supported(long, k, kr, v)
    assert not kd.expanded_attention_supported(long, k, None, v)


def test_expanded_without_channels():
    """Refused as any other width, by ValueError."""
    q, v, loc = torch.zeros(5, 2, 0, dtype=torch.bfloat16), torch.zeros(5, 2, 8, dtype=torch.bfloat16), torch.tensor([0, 5]).int()
    with pytest.raises(ValueError):
        kd.expanded_attention_fn(q, q, None, v, loc)


@pytest.mark.parametrize("dim,base,length", [(64, 1e4, 4096), (64, 1e4, 32768), (64, 1e4, 65536), (64, 1e4, 131072), (64, 1e4, 262144),
                                             (32, 1e4, 65536), (128, 1e6, 40960), (128, 5e5, 1 << 24), (64, 1e4, 200)])
@pytest.mark.parametrize("factor,fast,slow", [(4.0, 32.0, 1.0), (40.0, 32.0, 1.0), (8.0, 16.0, 2.0)])
def test_stretched_frequencies(dim, base, length, factor, fast, slow):
    """Each pair by itself: a frequency between base^(-2 i / dim) and that over the factor, by where
    the pair lies between those that would turn fast and slow times, which need not exist."""
    f, m = kd.rotary_frequencies(dim, base, factor=factor, original_length=length, beta_fast=fast, beta_slow=slow, device="cpu")

    def number(turns):  # of turns: base^(-2 i / dim) length / (2 pi) of pair i
        return dim / 2 * math.log(length / (2 * math.pi * turns)) / math.log(base)

    low, high = max(0, math.floor(number(fast))), math.ceil(number(slow))
    for i in range(dim // 2):
        plain = base ** (-2 * i / dim)
        part = min(1.0, max(0.0, (i - low) / (high - low)))
        want = plain * (1 - part) + plain / factor * part
        # FP64 to a few units in the last place, then one rounding to FP32.
        assert abs(f[i].item() - want) <= want * (2.0 ** -24 + 2.0 ** -48), (i, part)
        turns = plain * length / (2 * math.pi)
        if turns >= fast * (1 + 1e-12):
            assert f[i].item() == torch.tensor(plain).item()
        assert turns > slow or abs(f[i].item() * factor / plain - 1) < 2.0 ** -23
        assert turns <= slow * (1 + 1e-12) or f[i].item() > plain / factor  # it turns more often: not all divided
    assert m == 0.1 * math.log(factor) + 1


def test_rotary_units():
    """A workgroup counts a token's heads times other channels, and its threads' stride past them,
    in 31 bits: 49981 * 42966 is 2^31 - 2."""
    assert 49981 * 42966 == (1 << 31) - 2
    kw = dict(tokens=1, heads=49981, dim=42968, x1=42968, o1=42968, rotary=2, offset=0)
    assert rotary_code(**kw) == EUNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(s0=256, s1=16, pages=0), OK), (dict(s0=256, s1=0), EINVAL), (dict(s0=256, s1=15), EINVAL), (dict(s0=0, s1=16), EINVAL),
    (dict(s0=15, s1=9 * 16), EINVAL), (dict(s0=0, s1=0), EINVAL),
    # Strides of an axis of one entry mean nothing.
    (dict(s0=0, s1=15, pages=1), EINVAL), (dict(s0=15, s1=0, page=1), EINVAL), (dict(s0=0, s1=16, pages=0, page=1), OK),
])
def test_scales_that_overlap(kw, code):
    """Each token's scales are written, as its latent is: a broadcast cache of scales is refused."""
    assert write_code(cache=dict(e4m3=1, scales=A, **kw)) == code
