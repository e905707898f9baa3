"""Expanded attention at the ends of its arguments: scales of zero and next to it, heads far apart,
rows past 2^32 bytes, parts of the keys that weigh nothing."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from test_gpu_expanded_attention import BF16, DTYPES, F16, check, compare, inputs, normal, parts, run

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -140, 2.0 ** -160, -2.0 ** -160, 2.0 ** -1074])
@pytest.mark.parametrize("new,lens", [([70, 3], [70, 200]), ([300], [333]), ([40, 1], [5000, 900]), ([5, 3], [2, 0])])
def test_scale_zero(new, lens, scale, causal, dtype):
    """No score differs from another: the mean of the values that a row sees."""
    compare(inputs(new, lens, 2, 128, 64, 128, dtype), dtype, (new, scale), scale=scale, causal=causal)


def test_scale_zero_times_infinity():
    """0 times a score that is not finite is NaN, as in its definition: where the row sees it."""
    n = 100
    q, k, kr, v, loc, kv_loc = inputs([n], [n], 2, 64, 32, 64, BF16)
    clean = run((q, k, kr, v, loc, kv_loc), scale=0.0)
    k[40, 1, 3] = float("inf")
    got = run((q, k, kr, v, loc, kv_loc), scale=0.0)
    assert torch.equal(got[:40], clean[:40]) and torch.equal(got[:, 0], clean[:, 0])
    assert torch.isnan(got[40:, 1]).all()
    for value in (float("inf"), -float("inf"), float("nan")):
        bad = q.clone()
        bad[30, 0, 7] = value  # a channel of its own part, of head 0
        bad[31, 0, 70] = value
        got = run((bad, k, kr, v, loc, kv_loc), scale=0.0)[:40]
        assert torch.isnan(got[30:32, 0]).all()
        got[30:32, 0] = clean[30:32, 0]
        assert torch.equal(got, clean[:40])


@DTYPES
def test_heads_far_apart(dtype):
    """Head-major queries, keys and values: strides of heads past 2^23 elements."""
    heads, new, lens = 3, [5, 2], [65700, 100]
    q, k, kr, v, loc, kv_loc = inputs(new, lens, heads, 128, 64, 128, dtype)
    want = ref.expanded(q, k, kr, v, loc, kv_loc, 0.05)
    major = [torch.empty(heads, n, d, dtype=dtype, device="cuda").transpose(0, 1)
             for n, d in ((50000, 192), (sum(lens), 128), (sum(lens), 128))]
    major[0][:7].copy_(q)
    major[1].copy_(k)
    major[2].copy_(v)
    assert min(t.stride()[1] for t in major) >= 1 << 23
    out = torch.zeros(50000, heads, 128, dtype=dtype, device="cuda")
    kd.expanded_attention_fn(major[0], major[1], kr.cuda(), major[2], loc.cuda(), kv_loc.cuda(), scale=0.05, out=out)
    check(out[:7], want, dtype, v.double().abs().max(), "head-major")
    assert (out[7:] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weightless_parts(value):
    """Of a row's part of the keys only one is seen, with a score of -inf: its weight is 0, and 0
    times a value that is not finite is NaN."""
    new, lens = [100, 1], [150, 9000]  # 17 parts; the first sequence's hold a step of 64 keys or none
    assert parts(new, lens, 1)
    q, k, kr, v, loc, kv_loc = inputs(new, lens, 1, 128, 64, 128, BF16)
    q[..., 5] = -1.0
    for key in (64, 128):
        weak, bad = k.clone(), v.clone()
        weak[key, 0, 5] = float("inf")
        bad[key, 0, 7] = value
        want = run((q, weak, kr, v, loc, kv_loc))
        got = run((q, weak, kr, bad, loc, kv_loc))
        assert torch.isfinite(want).all()
        first = key - 50
        assert torch.isnan(got[first:100, 0, 7]).all() if value != value else not torch.isfinite(got[first:100, 0, 7]).any()
        got[first:100, 0, 7] = want[first:100, 0, 7]
        assert torch.equal(got, want), key


def test_rows_past_4_gb():
    """Keys and values at the largest stride of tokens: the last ones lie past 2^32 bytes."""
    n, stride = 300, (1 << 23) - 8  # elements, 16 MB
    assert (n - 1) * stride * 2 > 1 << 32
    buf = torch.empty((n - 1) * stride + 256, dtype=BF16, device="cuda")
    q, k, kr, v, loc, kv_loc = inputs([n], [n], 1, 128, 64, 128, BF16)
    far = buf.as_strided((n, 1, 256), (stride, 256, 1))
    far[..., :128].copy_(k)
    far[..., 128:].copy_(v)
    got = kd.expanded_attention_fn(q.cuda(), far[..., :128], kr.cuda(), far[..., 128:], loc.cuda())
    assert torch.equal(got, run((q, k, kr, v, loc, kv_loc)))
