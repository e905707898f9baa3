"""Long sequences in both forms against FP64, by the norm of each row's error: no step of keys is
lost or taken twice, in no worker's part and in no join (test_attention_error shows that the
bound would see it)."""

import pytest
import torch

import attention_error as ae
import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
#: Scores that differ little, so that every key weighs, and ordinary ones.
SCALES = pytest.mark.parametrize("scale", [0.02, 192 ** -0.5], ids=["flat", "ordinary"])


def normal(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@DTYPES
@SCALES
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,lens,heads,latent", [
    ([1], [20000], 12, 256), ([1, 1, 1], [5000, 3, 9000], 3, 256), ([1] * 7, [4000] * 7, 12, 512), ([1], [16000], 40, 384),
    ([3, 20], [9000, 4000], 12, 256), ([9, 1], [2000, 9000], 4, 512), ([1] * 37, [64 * i + 5 for i in range(37)], 12, 256)])
def test_absorbed(new, lens, heads, latent, e4m3, scale, dtype):
    table, pages = ref.tables(lens, 64)
    cache = ref.cache(pages, 64, latent, 64, dtype, e4m3)
    q, r = normal(sum(new), heads, latent, seed=1, dtype=dtype), normal(sum(new), heads, 64, seed=2, dtype=dtype)
    args = (q, r, cache, table, torch.tensor(lens, dtype=torch.int32), ref.starts(new))
    out, spread = ae.absorbed(*args, scale)
    got = kd.latent_attention_fn(*ref.on_gpu(q, r, *cache, *args[3:]), scale=scale)
    assert torch.isfinite(got).all()
    assert ae.worst(got, out, spread, dtype) < 1


@DTYPES
@SCALES
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,heads", [
    ([1], [5000], 2), ([33, 1, 0, 128, 7], [5000, 1, 0, 900, 64], 3), ([300], [6000], 3), ([400, 300], [400, 7000], 1),
    ([2, 40], [9000, 3000], 2), ([2000], [2500], 2)])
def test_expanded(new, lens, heads, causal, scale, dtype):
    q = normal(sum(new), heads, 192, seed=1, dtype=dtype)
    k, v = normal(sum(lens), heads, 128, seed=2, dtype=dtype), normal(sum(lens), heads, 128, seed=3, dtype=dtype)
    kr = normal(sum(lens), 64, seed=4, dtype=dtype)
    args = (q, k, kr, v, ref.starts(new), ref.starts(lens))
    out, spread = ae.expanded(*args, scale, causal)
    got = kd.expanded_attention_fn(*ref.on_gpu(*args), scale=scale, causal=causal)
    assert torch.isfinite(got).all()
    assert ae.worst(got, out, spread, dtype) < 1


@DTYPES
@pytest.mark.parametrize("e4m3", [False, True])
def test_wide_table(e4m3, dtype):
    """A table so wide that its keys could be 2^30 a sequence: the line of work counts several
    steps a unit. One row of it serves all sequences (a stride of 0)."""
    page, width, used = 128, 1 << 23, 70
    cache = ref.cache(used, page, 256, 64, dtype, e4m3)
    order = torch.randperm(used, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    wide = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    wide[0, :used] = order.cuda()
    for new, lens in (([1] * 100, [1 + 37 * i % 300 for i in range(99)] + [8900]), ([3, 1, 40] * 12, [8000, 1, 64] * 12),
                      ([1] * 300, [8960] + [5 * i for i in range(299)])):
        q, r = normal(sum(new), 12, 256, seed=1, dtype=dtype), normal(sum(new), 12, 64, seed=2, dtype=dtype)
        args = (torch.tensor(lens, dtype=torch.int32), ref.starts(new))
        out, spread = ae.absorbed(q, r, cache, order.expand(len(new), used), *args, 0.02)
        gpu = ref.on_gpu(q, r, *cache)
        got = kd.latent_attention_fn(*gpu, wide.expand(len(new), width), *(t.cuda() for t in args), scale=0.02)
        assert ae.worst(got, out, spread, dtype) < 1, lens[:3]
