"""Absorbed latent attention at the ends of its arguments."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from test_gpu_latent_not_finite import DTYPES, inputs

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -140, -2.0 ** -160])
def test_scale_zero(scale, dtype):
    """No score differs from another: the mean of the latents that a row sees."""
    args = inputs([3, 1, 2], [70, 3000, 1], 12, dtype)
    q, r, cache, table, lens, loc = args
    got = kd.latent_attention_fn(*ref.on_gpu(q, r, *cache, table, lens, loc), scale=scale)
    want = ref.attention(q, r, *cache, table, lens, loc, scale)
    half = torch.finfo(dtype).eps / 2
    err = (got.double().cpu() - want).abs()
    # Equal weights of 1 are exact: FP32 sums of up to 3000 terms, then one rounding.
    assert bool((err <= half * want.abs() + 3000 * 2.0 ** -24 * ref.values(*cache)[0].abs().max()).all())
