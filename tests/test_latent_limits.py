"""Limits of the latent attention operators on the host: what is refused, and what is not."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from packed_varlen_causal_depthwise_amd._lib import EUNSUPPORTED, OK
from test_latent_boundary import expanded_code

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
