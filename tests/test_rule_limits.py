"""Sizes and strides at which the gated delta rule and the norms refuse a call, on the host."""

import pytest

from packed_varlen_causal_depthwise_amd import _lib
from test_rule_boundary import A, EINVAL, EUNSUPPORTED, OK, pack


def prefill(**kw):
    return _lib.load().kdaconv_gated_delta_rule_validate(pack(**kw), 0, A, 1 << 50)


def update(n, **kw):
    return _lib.load().kdaconv_gated_delta_rule_validate(pack(T=n, S=n, **kw), 1, None, 0)


@pytest.mark.parametrize("tokens", [5, 17, 1000, 1 << 20])
def test_many_sequences_of_few_tokens(tokens):
    """A prefill launches a workgroup per sequence and head for the short ones: as many as an
    update may."""
    assert prefill(T=tokens, S=(1 << 23) - 1, H=1, HK=1) == OK
    assert prefill(T=tokens, S=1 << 23, H=1, HK=1) == EUNSUPPORTED
    assert prefill(T=tokens, S=1 << 25, H=1, HK=1) == EUNSUPPORTED
    assert prefill(T=tokens, S=1 << 20, H=8, HK=1) == EUNSUPPORTED
    assert update((1 << 23) - 1, H=1, HK=1) == OK
    assert update(1 << 23, H=1, HK=1) == EUNSUPPORTED


def test_many_tokens_of_few_sequences():
    """A workgroup per chunk of 32 tokens and head, and one per sequence and head."""
    assert prefill(T=131072, S=1, H=64, HK=64) == OK
    assert prefill(T=131072, S=1 << 16, H=64, HK=64) == OK
    assert prefill(T=1 << 22, S=1, H=63, HK=63) == OK
    assert prefill(T=1 << 22, S=1, H=64, HK=64) == EUNSUPPORTED


@pytest.mark.parametrize("axis,alone", [(("qs0", "ks0", "vs0", "gs0", "bs0"), dict(T=1)),
                                        (("qs1", "ks1"), dict(HK=1)),
                                        (("vs1", "gs1", "bs1"), dict(H=1, HK=1))])
def test_strides_of_an_axis_of_one_are_not_looked_at(axis, alone):
    for name in axis:
        for stride, code in ((1 << 23, EUNSUPPORTED), (-1, EUNSUPPORTED), ((1 << 23) - 1, OK)):
            assert prefill(**{name: stride}) == code
            assert update(100, **{name: stride}) == code
        for stride in (1 << 40, -1):
            kw = {**alone, name: stride}
            assert prefill(**{"S": 1, **kw}) == OK
            tokens = kw.pop("T", 100)
            assert update(tokens, **kw) == OK


def test_gated_norm_rows():
    """2^28 - 15 rows of 512 channels, 16 to a workgroup of 256, would be 2^32 threads."""
    gated = _lib.load().kdaconv_gated_rms_norm
    for tokens, heads in (((1 << 28) - 15, 1), (1, 1 << 28), (1 << 14, 1 << 14)):
        assert gated(A, _lib.BF16, tokens, heads, 512, 0, 0, A, 0, 0, 1, A, 1e-5, A, None) == EUNSUPPORTED
