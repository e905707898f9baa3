"""Absorbed latent attention over the paged cache against its definition in FP64."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def normal(*shape, seed=0, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def check(got, want, dtype, largest, what):
    """Elements of a convex combination of values up to `largest` (per row, broadcast).

    A weight's rounding to `dtype` is off by half a step h of it, and so is each term of the sum:
    h times the mean magnitude, at most h * largest in all. The sum of weights is taken before
    their rounding, in FP32. A score of up to 600 products summed in FP32 is off by 2^-24 times
    their number and size at the very most; with scores of size about 10 and less that is below
    2^-12 of a power of two, and so is exp2 of it. The result rounds once more.
    """
    half = torch.finfo(dtype).eps / 2
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = (got - want).abs()
    bad = err > half * want.abs() + (half + 2.0 ** -12) * largest + tiny
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(err / largest).max():.3g} of the values"


def inputs(new, lens, heads, latent, rope, page, dtype, e4m3=False, seed=0, width=None, head_major=False):
    """(q_latent, q_rope, cache, table, seq_lens, loc) on the CPU."""
    table, pages = ref.tables(lens, page, seed, width=width)
    cache = ref.cache(pages, page, latent, rope, dtype, e4m3, seed, one_tensor=not e4m3)
    tokens = sum(new)
    if head_major:
        ql = normal(heads, tokens, latent, seed=seed + 1, dtype=dtype).transpose(0, 1)
    else:
        ql = normal(tokens, heads, latent + 5, seed=seed + 1, dtype=dtype)[..., 3:3 + latent]
    qr = normal(tokens, heads, 7 + rope, seed=seed + 2, dtype=dtype)[..., 7:]
    return ql, qr, cache, table, torch.tensor(lens, dtype=torch.int32), ref.starts(new)


def run(args, scale, update=False, out=None):
    ql, qr, cache, table, lens, loc = args
    gpu = ref.on_gpu(ql, qr, *cache, table, lens, loc)
    if update:
        return kd.latent_attention_update(*gpu[:7], scale=scale, out=out)
    return kd.latent_attention_fn(*gpu, scale=scale, out=out)


def largest_of(cache):
    return ref.values(*cache)[0].abs().max()


def compare(args, scale, dtype, what, update=False):
    ql, qr, cache, table, lens, loc = args
    want = ref.attention(ql, qr, *cache, table, lens, loc, scale)
    check(run(args, scale, update), want, dtype, largest_of(cache), what)


DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=str)


@DTYPES
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads", [1, 12, 16, 17, 32, 64, 128])
def test_update_heads(heads, e4m3, dtype):
    lens = [1, 31, 32, 33, 127, 128, 129, 500, 1000]
    args = inputs([1] * len(lens), lens, heads, 512, 64, 16, dtype, e4m3, head_major=True)
    compare(args, 192 ** -0.5, dtype, heads, update=True)


@DTYPES
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("latent,rope,page", [(512, 64, 1), (256, 64, 64), (384, 32, 48), (128, 0, 7), (32, 8, 128),
                                              (416, 56, 5), (8, 16, 16)])
def test_update_sizes(latent, rope, page, e4m3, dtype):
    if e4m3 and latent % 32:
        pytest.skip("8-bit latents come in blocks of 32")
    args = inputs([1] * 5, [300, 1, 64, 65, 700], 12, latent, rope, page, dtype, e4m3)
    compare(args, (latent + rope) ** -0.5, dtype, (latent, rope, page), update=True)


@DTYPES
@pytest.mark.parametrize("heads", [3, 12])
@pytest.mark.parametrize("lens", [[20000], [5000, 3, 9000], [4000] * 7, [50] * 300, [1] * 520])
def test_update_split(lens, heads, dtype):
    """Sequences over many workers, workers over many sequences, a page table wider than needed."""
    args = inputs([1] * len(lens), lens, heads, 256, 64, 64, dtype, e4m3=len(lens) == 3, width=330)
    compare(args, 192 ** -0.5, dtype, lens[:3], update=True)


@DTYPES
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,lens,heads", [
    ([1, 2, 3, 4], [100, 2, 77, 1000], 8), ([5, 1, 0, 40, 9], [5, 700, 3, 41, 333], 4), ([130], [130], 2),
    ([33, 7], [400, 2000], 12), ([64] * 3, [64, 65, 3000], 1), ([3] * 90, [200] * 90, 12), ([2] * 5, [40, 2, 3, 900, 64], 12)])
def test_chunks(new, lens, heads, e4m3, dtype):
    args = inputs(new, lens, heads, 512, 64, 16, dtype, e4m3)
    compare(args, 192 ** -0.5, dtype, new)


def test_rows_without_tokens():
    """Sequences with fewer cached than new tokens, none at all, pages outside the cache, rows
    that no sequence owns."""
    new, lens = [4, 3, 2, 2, 1], [2, 0, 100, 40, 64]
    ql, qr, cache, table, seq_lens, loc = inputs(new, [2, 0, 100, 40, 64], 5, 256, 32, 16, BF16, width=9)
    table[2, 1], table[2, 3] = -1, cache[0].shape[0]
    table[3, :] = 1 << 20  # nothing left
    seq_lens = torch.tensor([2, -7, 100, 40, 1000], dtype=torch.int32)  # the last past its table
    want = ref.attention(ql, qr, *cache, table, torch.tensor([2, 0, 100, 40, 144]), loc, 0.1)
    # (the definition, too: 144 is the table's width; row 0 of the last sequence sees 1000 - 1 + 1)
    out = torch.full((ql.shape[0] + 2, 5, 256), 7.0, dtype=BF16, device="cuda")
    pad = [torch.cat([t, t[:2]]) for t in (ql, qr)]
    got = run((*pad, cache, table, seq_lens, loc), 0.1, out=out)
    assert (got[-2:] == 7).all()
    check(got[:-2], want, BF16, largest_of(cache), "rows")
    assert (got[:2] == 0).all() and (got[4:7] == 0).all() and (got[9:11] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_memory_nobody_owns_is_not_used(e4m3):
    """NaN in all slots that no sequence reaches: ends of pages, other pages, other tokens."""
    new, lens, page = [1, 3, 1], [37, 70, 5], 32
    ql, qr, cache, table, seq_lens, loc = inputs(new, lens, 12, 512, 64, page, BF16, e4m3)
    used = torch.cat([ref.slots_of(table[s], n, page, cache[0].shape[0]) for s, n in enumerate(lens)])
    free = torch.ones(cache[0].shape[0] * page, dtype=torch.bool)
    free[used] = False
    lat, rop = cache[0].clone(), cache[1].clone()
    want = run((ql, qr, cache, table, seq_lens, loc), 0.1)
    if e4m3:
        lat.view(torch.uint8).flatten(0, 1)[free] = 0x7F
    else:
        lat.flatten(0, 1)[free] = float("nan")
    rop.flatten(0, 1)[free] = float("nan")
    got = run((ql, qr, (lat, rop, cache[2]), table, seq_lens, loc), 0.1)
    assert torch.isfinite(got).all() and torch.equal(got, want)


@DTYPES
def test_large_scores(dtype):
    """Scores far apart and far from zero: the softmax picks one token; sums are rescaled on the
    way as the largest score grows along the keys."""
    n = 300
    ql, qr, cache, table, seq_lens, loc = inputs([1], [n], 16, 256, 64, 16, dtype)
    at = ref.slots_of(table[0], n, 16, cache[0].shape[0])
    lat, rop = cache[0].clone(), cache[1].clone()
    ramp = torch.arange(n).double() - 150
    rop.flatten(0, 1)[at] = 0
    rop.flatten(0, 1)[at, 0] = ramp.to(dtype)
    qr = torch.zeros_like(qr)
    qr[..., 0] = 8.0  # scores rise by 8 * 0.5 a token, over 1200 in all; the latents add a few
    args = (ql, qr, (lat, rop, None), table, seq_lens, loc)
    # FP32 sums of size 1200 are off by 2^-14 or so, and so are weights: 2^-12 covers both
    compare(args, 0.5, dtype, "rising")
    rop.flatten(0, 1)[at, 0] = -ramp.to(dtype)
    compare((ql, qr, (lat, rop, None), table, seq_lens, loc), 0.5, dtype, "falling")


def test_values_that_are_not_finite():
    """A NaN reaches the rows that see its token, no other."""
    new, lens, page = [6, 1], [40, 64], 16
    ql, qr, cache, table, seq_lens, loc = inputs(new, lens, 3, 256, 64, page, BF16)
    lat = cache[0].clone()
    at = ref.slots_of(table[0], 40, page, lat.shape[0])
    lat.flatten(0, 1)[at[37], 5] = float("nan")  # tokens 3, 4 and 5 of 6 see it
    got = run((ql, qr, (lat, cache[1], None), table, seq_lens, loc), 0.1)
    want = run((ql, qr, cache, table, seq_lens, loc), 0.1)
    assert torch.equal(got[:3], want[:3]) and torch.equal(got[6], want[6])
    assert torch.isnan(got[3:6]).all()


def test_update_is_the_chunk_of_one():
    lens = [5, 900, 64]
    args = inputs([1] * 3, lens, 12, 512, 64, 16, BF16)
    assert torch.equal(run(args, 0.1), run(args, 0.1, update=True))


def test_graph_and_two_at_once():
    """A captured step replayed on other lengths, pages and queries, beside eager calls on
    another stream."""
    lens = [900, 64, 1, 2000]
    ql, qr, cache, table, seq_lens, loc = inputs([1] * 4, lens, 12, 512, 64, 64, BF16)
    gpu = ref.on_gpu(ql, qr, *cache, table, seq_lens)
    other = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = kd.latent_attention_update(*gpu, scale=0.1)
    for seed, change in ((5, [900, 64, 1, 2000]), (6, [10, 0, 64, 1999]), (7, [513, 33, 2, 128])):
        gpu[0].copy_(normal(*ql.shape, seed=seed, dtype=BF16))
        gpu[6].copy_(torch.tensor(change, dtype=torch.int32))
        want = kd.latent_attention_update(*gpu, scale=0.1)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            again = [kd.latent_attention_update(*gpu, scale=0.1) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(a, want) for a in again)
        check(want, ref.attention(gpu[0].cpu(), qr, *cache, table, torch.tensor(change), loc, 0.1), BF16,
              largest_of(cache), change)


def test_far_pages():
    """A cache whose last page lies past 2^32 bytes."""
    pages, page = 140, 64
    big = torch.empty(pages, 16 * 1024 * 1024, dtype=BF16, device="cuda")  # 32 MB a page, 4.4 GB
    both = big[:, : page * 320].unflatten(1, (page, 320))
    small = normal(pages, page, 320, seed=3, dtype=BF16)
    both.copy_(small)
    lens = [150, 64]
    table = torch.tensor([[139, 0, 138], [137, 5, 5]], dtype=torch.int32)
    ql, qr = normal(2, 4, 256, seed=4, dtype=BF16), normal(2, 4, 64, seed=5, dtype=BF16)
    got = kd.latent_attention_update(ql.cuda(), qr.cuda(), both[..., :256], both[..., 256:], None, table.cuda(),
                                     torch.tensor(lens, dtype=torch.int32).cuda(), scale=0.1)
    want = ref.attention(ql, qr, small[..., :256], small[..., 256:], None, table, lens, ref.starts([1, 1]), 0.1)
    check(got, want, BF16, small.double().abs().max(), "far")
    out = kd.latent_cache_read(both[..., :256], both[..., 256:], None, table.cuda(), ref.starts(lens).cuda(), 214)
    at = torch.cat([ref.slots_of(table[s], n, page, pages) for s, n in enumerate(lens)])
    assert torch.equal(out.cpu(), small.flatten(0, 1)[at])


def test_empty():
    ql, qr, cache, table, lens, loc = inputs([1], [5], 2, 64, 8, 4, BF16)
    g = ref.on_gpu(ql, qr, *cache, table, lens, loc)
    assert kd.latent_attention_update(g[0][:0], g[1][:0], *g[2:7], scale=1.0).shape == (0, 2, 64)
    assert kd.latent_attention_fn(g[0][:0], g[1][:0], *g[2:7], g[7][:1], scale=1.0).shape == (0, 2, 64)
    assert kd.latent_attention_supported(*g[:5]) and not kd.latent_attention_supported(ql, qr, *cache)


@pytest.mark.parametrize("latent", [512, 480, 256])
def test_scales_at_odd_addresses(latent):
    """Scales that lie at no multiple of anything, among other bytes."""
    lens = [70, 3, 200]
    table, pages = ref.tables(lens, 8)
    c, r, s = ref.on_gpu(*ref.cache(pages, 8, latent, 64, torch.bfloat16, e4m3=True))
    among = torch.full((pages, 8, latent // 32 + 3), 255, dtype=torch.uint8, device="cuda")
    odd = among[..., 1:1 + latent // 32]
    odd.copy_(s)
    g = torch.Generator().manual_seed(3)
    for heads in (12, 40):
        q = torch.randn(3, heads, latent, generator=g).bfloat16().cuda()
        qr = torch.randn(3, heads, 64, generator=g).bfloat16().cuda()
        rest = (table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        want = kd.latent_attention_update(q, qr, c, r, s, *rest, scale=0.05)
        assert torch.isfinite(want).all()
        assert torch.equal(kd.latent_attention_update(q, qr, c, r, odd, *rest, scale=0.05), want)
