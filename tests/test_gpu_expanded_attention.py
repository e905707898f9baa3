"""Expanded attention of packed sequences against its definition in FP64."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from packed_varlen_causal_depthwise_amd import _lib

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=str)


def normal(*shape, seed=0, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def check(got, want, dtype, largest, what):
    """Elements of a convex combination of values up to `largest`. A weight rounded to `dtype` is
    off by half a step h of it, so the sum by at most h * largest; scores below 16 in size, sums
    of up to 192 FP32 products, leave the weights within 2^-12; the result rounds once more."""
    half = torch.finfo(dtype).eps / 2
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = (got - want).abs()
    bad = err > half * want.abs() + (half + 2.0 ** -12) * largest + tiny
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(err / largest).max():.3g} of the values"


def inputs(new, lens, heads, dim, rope, vdim, dtype, seed=0):
    """(q, k, k_rope, v, loc, kv_loc) on the CPU; k and v slices of one tensor where they can be."""
    T, M = sum(new), sum(lens)
    q = normal(T, heads, dim + rope + 3, seed=seed + 1, dtype=dtype)[..., 1:1 + dim + rope]
    kv = normal(M, heads, dim + vdim, seed=seed + 2, dtype=dtype)
    kr = normal(M, 64 + rope, seed=seed + 3, dtype=dtype)[:, 64:] if rope else None
    return q, kv[..., :dim], kr, kv[..., dim:], ref.starts(new), ref.starts(lens)


def run(args, out=None, **kw):
    return kd.expanded_attention_fn(*ref.on_gpu(*args), out=out, **kw)


def compare(args, dtype, what, scale=None, causal=True):
    q, k, kr, v, loc, kv_loc = args
    s = q.shape[2] ** -0.5 if scale is None else scale
    want = ref.expanded(*args, s, causal)
    check(run(args, scale=scale, causal=causal), want, dtype, v.double().abs().max(), what)


@DTYPES
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_one_prompt(n, dtype):
    compare(inputs([n], [n], 2, 128, 64, 128, dtype), dtype, n)


@DTYPES
@pytest.mark.parametrize("dim,rope,vdim", [(128, 64, 128), (64, 64, 64), (128, 32, 128), (64, 32, 64), (128, 0, 128),
                                           (8, 8, 8), (96, 48, 72), (40, 0, 104), (120, 56, 64), (64, 16, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_sizes(dim, rope, vdim, causal, dtype):
    compare(inputs([70, 3], [70, 200], 3, dim, rope, vdim, dtype), dtype, (dim, rope, vdim), causal=causal)
    compare(inputs([300], [333], 1, dim, rope, vdim, dtype), dtype, (dim, rope, vdim), causal=causal)


@DTYPES
@pytest.mark.parametrize("new,lens,heads", [
    ([1, 2, 0, 130, 5], [9, 2, 0, 130, 1000], 4), ([64] * 70, [64] * 70, 1), ([1] * 300, [3] * 300, 2),
    ([1000, 17], [1000, 4000], 2), ([513, 300, 260], [600, 300, 900], 3), ([2, 0, 0, 0, 1], [2, 0, 5, 0, 70], 12)])
def test_batches(new, lens, heads, dtype):
    compare(inputs(new, lens, heads, 128, 64, 128, dtype), dtype, new[:4])


def test_rows_without_keys():
    """More queries than keys, no keys at all, rows that no sequence owns."""
    new, lens = [5, 3, 200], [2, 0, 150]
    q, k, kr, v, loc, kv_loc = inputs(new, lens, 2, 64, 32, 64, BF16)
    want = ref.expanded(q, k, kr, v, loc, kv_loc, 0.1)
    out = torch.full((q.shape[0] + 3, 2, 64), 7.0, dtype=BF16, device="cuda")
    pad = torch.cat([q[:2], q, q[:1]])
    got = run((pad, k, kr, v, loc + 2, kv_loc), out=out, scale=0.1)
    assert (got[:2] == 7).all() and (got[-1:] == 7).all()
    check(got[2:-1], want, BF16, v.double().abs().max(), "rows")
    assert (got[2:5] == 0).all() and (got[7:60] == 0).all()
    none = run((q[:4], k[:0], kr[:0], v[:0], ref.starts([4]), ref.starts([0])), scale=0.1)
    assert (none == 0).all()


def test_memory_nobody_owns_is_not_used():
    """NaN around the keys of every sequence, and in queries of others."""
    new, lens = [40, 3], [40, 100]
    q, k, kr, v, loc, kv_loc = inputs(new, lens, 2, 128, 64, 128, BF16)
    want = run((q, k, kr, v, loc, kv_loc))
    nan = float("nan")

    def spread(t, gap):
        big = torch.full((t.shape[0] + 3 * gap, *t.shape[1:]), nan, dtype=t.dtype)
        big[gap:gap + 40], big[2 * gap + 40:2 * gap + 40 + t.shape[0] - 40] = t[:40], t[40:]
        return big

    gap = 70
    far = (spread(q, 8), spread(k, gap), spread(kr, gap), spread(v, gap))
    for first in (0, 1):  # sequences apart: each alone
        a, b = int(loc[first]), int(loc[first + 1])
        c, d = int(kv_loc[first]), int(kv_loc[first + 1])
        ql = torch.tensor([a + 8 * (first + 1), b + 8 * (first + 1)], dtype=torch.int32)
        kl = torch.tensor([c + gap * (first + 1), d + gap * (first + 1)], dtype=torch.int32)
        out = torch.zeros(far[0].shape[0], 2, 128, dtype=BF16, device="cuda")
        got = run((*far, ql, kl), out=out)
        assert torch.equal(got[int(ql[0]):int(ql[1])], want[a:b])


@DTYPES
@pytest.mark.parametrize("scale", [2.0, -2.0])
def test_large_scores(scale, dtype):
    """Scores that rise or fall along the keys, 700 in all: sums are rescaled on the way."""
    n = 350
    q, k, kr, v, loc, kv_loc = inputs([n], [n], 1, 64, 32, 64, dtype)
    q, k, kr = torch.zeros_like(q), torch.zeros_like(k), kr * 0
    q[..., 0] = 1.0
    k[:, 0, 0] = (torch.arange(n) - 175).to(dtype)  # exact
    q[..., 70], kr[:, 6] = 0.5, normal(n, seed=9, dtype=dtype)
    # scores of size 350 in steps of 2^-15: weights within 2^-14
    compare((q, k, kr, v, loc, kv_loc), dtype, scale, scale=scale)


def test_values_that_are_not_finite():
    """A NaN in a key or a value, an infinity in a value: no row that does not see it."""
    n = 300
    q, k, kr, v, loc, kv_loc = inputs([n], [n], 2, 128, 64, 128, BF16)
    clean = run((q, k, kr, v, loc, kv_loc))
    for at in (0, 37, 130, 299):
        for what in ("k", "r", "v", "inf"):
            t = {"k": k, "r": kr, "v": v, "inf": v}[what].clone()
            if what == "r":
                t[at, 5] = float("nan")
            else:
                t[at, 1, 5] = float("inf") if what == "inf" else float("nan")
            args = [q, k, kr, v, loc, kv_loc]
            args[{"k": 1, "r": 2, "v": 3, "inf": 3}[what]] = t
            got = run(args)
            assert torch.equal(got[:at], clean[:at]), (at, what)
            if what == "r":
                assert torch.isnan(got[at:]).all()
            elif what == "k":
                assert torch.isnan(got[at:, 1]).all() and torch.equal(got[:, 0], clean[:, 0])
            else:  # only that channel of that head
                assert not torch.isfinite(got[at:, 1, 5]).any()
                got[at:, 1, 5] = clean[at:, 1, 5]
                assert torch.equal(got, clean), (at, what)


def test_far_rows():
    """Keys and values past 2^32 bytes."""
    n, stride = 300, 1 << 23
    buf = torch.empty(n * stride // 2 + 512, dtype=BF16, device="cuda")  # rows 8 MB apart: 2.5 GB
    q, k, kr, v, loc, kv_loc = inputs([n], [n], 1, 128, 64, 128, BF16)
    far = buf.as_strided((n, 1, 256), (stride // 2, 256, 1))
    far[..., :128].copy_(k)
    far[..., 128:].copy_(v)
    got = kd.expanded_attention_fn(q.cuda(), far[..., :128], kr.cuda(), far[..., 128:], loc.cuda())
    assert torch.equal(got, run((q, k, kr, v, loc, kv_loc)))


def test_graph_and_streams():
    new = [200, 1, 90]
    args = ref.on_gpu(*inputs(new, new, 4, 128, 64, 128, BF16))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = kd.expanded_attention_fn(*args)
    for seed, change in ((4, new), (5, [1, 290, 0]), (6, [97, 97, 97])):
        args[0].copy_(normal(*args[0].shape, seed=seed, dtype=BF16))
        for loc in args[4:]:
            loc.copy_(ref.starts(change))
        want = kd.expanded_attention_fn(*args)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            again = [kd.expanded_attention_fn(*args) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(a, want) for a in again)


def test_empty():
    q, k, kr, v, loc, kv_loc = ref.on_gpu(*inputs([3], [3], 2, 64, 32, 64, BF16))
    assert kd.expanded_attention_fn(q[:0], k, kr, v, loc, kv_loc).shape == (0, 2, 64)
    assert kd.expanded_attention_fn(q, k, kr, v, loc[:1], kv_loc[:1]).shape == (3, 2, 64)
    assert kd.expanded_attention_supported(q, k, kr, v) and not kd.expanded_attention_supported(q.cpu(), k, kr, v)


def parts(new, lens, heads):
    """Whether the call splits its keys."""
    return _lib.load().kdaconv_expanded_attention_workspace(sum(new), sum(lens), len(new), heads, 64) > 0


@DTYPES
@pytest.mark.parametrize("new,lens,heads,sizes", [
    ([1], [5000], 2, (128, 64, 128)), ([1], [513], 1, (8, 8, 8)), ([33, 1, 0, 128, 7], [5000, 1, 0, 900, 64], 3, (128, 64, 128)),
    ([300], [6000], 3, (128, 32, 128)), ([400, 300], [400, 7000], 1, (64, 64, 64)), ([129] * 3, [1100, 130, 3000], 4, (40, 0, 104)),
    ([90, 5], [60, 2000], 2, (64, 32, 64)), ([2] * 60, [700] * 60, 2, (64, 16, 32))])
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows_over_many_keys(new, lens, heads, sizes, causal, dtype):
    """Keys split among workgroups: parts that end inside a block's reach, or see nothing."""
    assert parts(new, lens, heads)
    compare(inputs(new, lens, heads, *sizes, dtype), dtype, (new, lens), causal=causal)


def test_split_rows_without_keys():
    new, lens = [5, 3, 40, 2], [2, 0, 5000, 0]
    assert parts(new, lens, 2)
    q, k, kr, v, loc, kv_loc = inputs(new, lens, 2, 64, 32, 64, BF16)
    out = torch.full((q.shape[0] + 3, 2, 64), 7.0, dtype=BF16, device="cuda")
    got = run((torch.cat([q[:2], q, q[:1]]), k, kr, v, loc + 2, kv_loc), out=out, scale=0.1)
    assert (got[:2] == 7).all() and (got[-1:] == 7).all()
    check(got[2:-1], ref.expanded(q, k, kr, v, loc, kv_loc, 0.1), BF16, v.double().abs().max(), "rows")
    assert (got[2:5] == 0).all() and (got[7:10] == 0).all() and (got[50:52] == 0).all()


@DTYPES
@pytest.mark.parametrize("scale", [2.0, -2.0])
def test_split_large_scores(scale, dtype):
    """Scores that rise or fall by 700 along the keys: of most parts nothing is left."""
    m = 2100
    q, k, kr, v, loc, kv_loc = inputs([40], [m], 1, 64, 32, 64, dtype)
    q, k, kr = torch.zeros_like(q), torch.zeros_like(k), kr * 0
    q[..., 0] = 1.0
    k[:, 0, 0] = ((torch.arange(m) - m // 2) // 6).to(dtype)  # up to 175, exact
    q[..., 70], kr[:, 6] = 0.5, normal(m, seed=9, dtype=dtype)
    compare((q, k, kr, v, loc, kv_loc), dtype, scale, scale=scale)


def test_split_values_that_are_not_finite():
    """In parts before, at and behind what rows see."""
    n, m = 70, 3000
    assert parts([n], [m], 2)
    q, k, kr, v, loc, kv_loc = inputs([n], [m], 2, 128, 64, 128, BF16)
    clean = run((q, k, kr, v, loc, kv_loc))
    for key in (0, 1000, 2929, 2930, 2931, 2960, 2999):
        at = max(0, key - (m - n))  # the first row that sees it
        for what in ("k", "v", "inf"):
            t = (k if what == "k" else v).clone()
            t[key, 1, 5] = float("inf") if what == "inf" else float("nan")
            got = run((q, t, kr, v, loc, kv_loc) if what == "k" else (q, k, kr, t, loc, kv_loc))
            assert torch.equal(got[:at], clean[:at]) and torch.equal(got[:, 0], clean[:, 0]), (key, what)
            if what == "k":
                assert torch.isnan(got[at:, 1]).all(), key
            else:
                assert not torch.isfinite(got[at:, 1, 5]).any(), (key, what)
                got[at:, 1, 5] = clean[at:, 1, 5]
                assert torch.equal(got, clean), (key, what)


def test_split_graph_and_streams():
    """Two captured calls and eager ones on another stream, each with scratch memory of its own."""
    new, lens = [20, 1], [2000, 600]
    assert parts(new, lens, 4)
    args = ref.on_gpu(*inputs(new, lens, 4, 128, 64, 128, BF16))
    other = torch.cuda.Stream()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    torch.cuda.synchronize()
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(kd.expanded_attention_fn(*args))
    for seed, change, keys in ((4, new, lens), (5, [1, 20], [0, 2600]), (6, [10, 11], [1300, 1300])):
        args[0].copy_(normal(*args[0].shape, seed=seed, dtype=BF16))
        args[4].copy_(ref.starts(change))
        args[5].copy_(ref.starts(keys))
        want = kd.expanded_attention_fn(*args)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            graphs[1].replay()
            again = [kd.expanded_attention_fn(*args) for _ in range(3)]
        graphs[0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, want) for a in outs + again), seed
