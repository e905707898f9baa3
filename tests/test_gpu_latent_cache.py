"""Rotary positions and the latent cache's write and read, against FP64 (latent_reference)."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def normal(*shape, seed=0, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def close(got, want, dtype, slack, what):
    """Each element within half a step of `dtype` and `slack` (an absolute error, broadcast)."""
    got = got.double().cpu()
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    err = (got - want).abs()
    bad = err > half * want.abs() + slack * (1 + half) + tiny
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {err.max():.3g}"


def turn_slack(x, scale=1.0):
    """The arithmetic's part: an angle off by 2^-26 of a turn is 2 pi 2^-26 = 1.6 * 2^-24, sine
    and cosine 2 units of 2^-24 each, the factor, a product and a sum one each: below 7 * 2^-24
    of |u| + |v|, which is at most sqrt(2) times the pair's length."""
    return 10 * 2.0 ** -24 * scale * x.double().abs().amax(-1, keepdim=True) * 2 ** 0.5


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("tokens,heads,dim,rotary,offset", [
    (1, 1, 2, 2, 0), (1, 12, 192, 64, 128), (37, 12, 192, 64, 128), (3, 5, 70, 6, 33),
    (9, 1, 128, 128, 0), (5, 2, 200, 72, 40), (2100, 3, 96, 32, 64), (4, 2, 600, 512, 8),
    (33, 7, 24, 8, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(tokens, heads, dim, rotary, offset, interleaved, dtype):
    x = normal(tokens, heads, dim, seed=1, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=torch.Generator().manual_seed(2))
    f = ref.frequencies(rotary)
    want = x.double().clone()
    part = slice(offset, offset + rotary)
    want[..., part] = ref.turned(x[..., part], pos, f, interleaved, 1.25)
    kw = dict(offset=offset, interleaved=interleaved, scale=1.25)
    got = kd.rotary_embedding(x.cuda(), pos.cuda(), f.cuda(), **kw)
    close(got, want, dtype, turn_slack(x, 1.25), "new")
    y = x.cuda()
    assert kd.rotary_embedding(y, pos.to(torch.int32).cuda(), f.cuda(), out=y, **kw) is y
    assert torch.equal(y, got)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_strides(interleaved):
    rows = normal(50, 1001, seed=3, dtype=BF16).cuda()
    x = rows[:, 1:1 + 5 * 160].unflatten(1, (5, 160))[..., 3:99]
    pos, f = torch.arange(50).cuda(), ref.frequencies(64).cuda()
    want = kd.rotary_embedding(x.contiguous(), pos, f, offset=16, interleaved=interleaved)
    got = kd.rotary_embedding(x, pos, f, offset=16, interleaved=interleaved)
    assert torch.equal(got, want)
    keep = rows.clone()
    out = torch.zeros(5, 50, 96, device="cuda", dtype=BF16).transpose(0, 1)
    assert torch.equal(kd.rotary_embedding(x, pos, f, offset=16, interleaved=interleaved, out=out), want)
    assert torch.equal(rows, keep)
    kd.rotary_embedding(x, pos, f, offset=16, interleaved=interleaved, out=x)
    assert torch.equal(x, want)
    x.copy_(keep[:, 1:1 + 5 * 160].unflatten(1, (5, 160))[..., 3:99])
    assert torch.equal(rows, keep)  # nothing beside the view was written


def test_rotary_far_positions():
    """Angles of far and negative positions, against 300-bit arithmetic."""
    from mpmath import cos, mp, mpf, sin

    mp.prec = 300
    pos = torch.tensor([0, 1, -1, 12345678, 1 << 24, (1 << 29) - 1, -(1 << 29) + 1])
    f = ref.frequencies(32)
    x = torch.zeros(len(pos), 1, 32)
    x[..., :16] = 1.0
    got = kd.rotary_embedding(x.cuda(), pos.cuda(), f.cuda()).cpu().double()
    for i, p in enumerate(pos.tolist()):
        for j, w in enumerate(f.tolist()):
            a = mpf(p) * mpf(w)
            assert abs(float(cos(a)) - got[i, 0, j]) < 8 * 2.0 ** -24
            assert abs(float(sin(a)) - got[i, 0, 16 + j]) < 8 * 2.0 ** -24


def test_frequencies():
    f, s = kd.rotary_frequencies(64, device="cpu")
    assert s == 1.0 and torch.equal(f, ref.frequencies(64))
    g, s = kd.rotary_frequencies(64, factor=4.0, original_length=4096, device="cpu")
    assert abs(s - 1.1386294361119891) < 1e-12
    turns = 4096 * f.double() / (2 * torch.pi)
    assert torch.equal(g[turns > 64], f[turns > 64])
    assert torch.allclose(g[turns < 0.5], f[turns < 0.5] / 4) and (g <= f).all() and (g >= f / 4).all()


def write_case(tokens, latent, rope, page, dtype, e4m3, interleaved=False, one=False, seed=0):
    table, pages = ref.tables([tokens], page, seed)
    cache = ref.cache(pages, page, latent, rope, dtype, e4m3, seed, one)
    rows = normal(tokens, latent + rope + 3, seed=seed + 1, dtype=dtype)
    slots = ref.slots_of(table[0], tokens, page, pages)
    pos = torch.randint(0, 1 << 17, (tokens,), generator=torch.Generator().manual_seed(seed + 2))
    return rows[:, 1:1 + latent], rows[:, 1 + latent:1 + latent + rope], cache, slots, pos


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tokens,latent,rope,page", [
    (1, 512, 64, 16), (37, 512, 64, 64), (5, 32, 0, 1), (130, 384, 32, 48), (33, 256, 8, 7), (700, 512, 64, 100)])
def test_write(tokens, latent, rope, page, e4m3, dtype):
    for interleaved, norm in ((False, True), (True, False)):
        x, r, cache, slots, pos = write_case(tokens, latent, rope, page, dtype, e4m3, one=not e4m3)
        if tokens > 4:
            slots[3], slots[tokens // 2] = -1, 1 << 40
        w = 1 + 0.1 * normal(latent, seed=9)
        f = ref.frequencies(rope) if rope else torch.zeros(0)
        lat, rop, sc = ref.on_gpu(*cache)
        before = [None if t is None else t.view(torch.uint8).clone() for t in (lat, rop, sc)]
        kd.latent_cache_write(x.cuda(), r.cuda(), lat, rop, sc, slots.cuda(),
                              **(dict(weight=w.cuda(), eps=1e-6) if norm else {}),
                              positions=pos.cuda(), inv_freq=f.cuda(), interleaved=interleaved, rope_scale=1.5)
        live = (slots >= 0) & (slots < 1 << 30)
        at = slots[live]
        y = ref.normed(x, w, 1e-6)[live] if norm else x.double()[live]
        flat = [None if t is None else t.cpu().flatten(0, 1) for t in (lat, rop, sc)]
        if e4m3:
            v, bytes_ = ref.to_8_bits(y)
            assert torch.equal(flat[2][at], bytes_)
            assert torch.equal(flat[0][at].double(), v)
        else:
            close(flat[0][at], y, dtype, 2.0 ** -24 * y.abs(), "latents")  # y rounds to FP32 first
        if rope:
            close(flat[1][at], ref.turned(r[live][:, None], pos[live], f, interleaved, 1.5)[:, 0], dtype,
                  turn_slack(r[live], 1.5), "ropes")
        rest = torch.ones(lat.shape[0] * page, dtype=torch.bool)
        rest[at] = False
        for t, b in zip((lat, rop, sc), before):
            if t is not None and t.numel():
                assert torch.equal(t.view(torch.uint8).flatten(0, 1)[rest.cuda()], b.flatten(0, 1)[rest.cuda()])


def test_write_8_bit_borders():
    """Every border between codes, block maxima at powers of two and at 448 of them, zeros,
    subnormals, infinities and NaN, without the norm."""
    dtype = BF16
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2  # 5 significant bits: exact in bf16
    x = torch.zeros(64, 512, dtype=torch.float64)
    flat = torch.cat([codes, mid, -codes, -mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -7)])
    for i in range(64):
        scale = 2.0 ** (4 * (i - 32))
        x[i] = flat[(torch.arange(512) * 7 + i * 13) % len(flat)] * scale
        x[i, ::32] = (448.0, 449.0, 256.0, 448.0 * (1 + 2.0 ** -7))[i % 4] * scale
    x[5, :32] = 0.0
    x[6, 3], x[6, 40], x[6, 70] = float("inf"), float("nan"), -float("inf")
    x[7, :64] = 2.0 ** -126
    x[8] = 3e38
    x = x.to(dtype)
    lat, rop, sc = (t.cuda() for t in ref.cache(2, 32, 512, 0, dtype, True))
    kd.latent_cache_write(x.cuda(), torch.empty(64, 0, dtype=dtype).cuda(), lat, rop, sc, torch.arange(64).cuda())
    v, bytes_ = ref.to_8_bits(x)
    assert torch.equal(sc.cpu().flatten(0, 1), bytes_)
    got = lat.cpu().flatten(0, 1).double()
    assert torch.equal(torch.isnan(got), torch.isnan(v)) and torch.equal(got.nan_to_num(0), v.nan_to_num(0))


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lengths,page,latent,rope", [
    ([1], 1, 512, 64), ([0, 5, 0, 0, 70, 1, 0], 16, 512, 64), ([300, 41], 48, 384, 32),
    ([17] * 130, 64, 32, 0), ([64, 128, 1000], 64, 256, 8)])
def test_read(lengths, page, latent, rope, e4m3, dtype):
    table, pages = ref.tables(lengths, page)
    cache = ref.cache(pages, page, latent, rope, dtype, e4m3)
    c, r = ref.values(*cache)
    total, loc = sum(lengths), ref.starts(lengths)
    loc += 2  # rows before and after that no sequence owns
    out = torch.full((total + 5, latent + rope), 7.0, dtype=dtype, device="cuda")
    got = kd.latent_cache_read(*ref.on_gpu(*cache), table.cuda(), loc.cuda(), total + 5, out=out).cpu()
    assert (got[:2] == 7).all() and (got[total + 2:] == 7).all()
    at = torch.cat([ref.slots_of(table[s], n, page, pages) for s, n in enumerate(lengths)])
    want = torch.cat([c[at], r[at]], -1)
    close(got[2:total + 2], want, dtype, 0.0, "rows")


def test_read_pages_outside():
    lengths, page = [50, 40], 16
    table, pages = ref.tables(lengths, page)
    cache = ref.cache(pages, page, 64, 8, BF16)
    table[0, 1], table[1, 0] = -1, pages
    loc = ref.starts([70, 40])  # the first sequence goes past its table's columns
    got = kd.latent_cache_read(*ref.on_gpu(*cache), table.cuda(), loc.cuda(), 110).cpu()
    c, r = ref.values(*cache)
    both = torch.cat([c, r], -1)
    for s, (a, n) in enumerate(((0, 70), (70, 40))):
        at = ref.slots_of(table[s], n, page, pages)
        want = torch.where(at[:, None] >= 0, both[at.clamp(min=0)], 0.0)
        assert torch.equal(got[a:a + n].double(), want)


def test_write_then_read_in_a_graph():
    x, r, cache, slots, pos = write_case(200, 512, 64, 32, BF16, True)
    lat, rop, sc = (t.cuda() for t in cache)
    x, r, slots, pos = x.cuda(), r.cuda(), slots.cuda(), pos.cuda()
    table = torch.arange(lat.shape[0], dtype=torch.int32, device="cuda")[None]
    loc = torch.tensor([0, lat.shape[0] * 32], dtype=torch.int32, device="cuda")
    f = ref.frequencies(64).cuda()

    def both():
        kd.rotary_embedding(r[:, None], pos, f, out=r[:, None])
        kd.latent_cache_write(x, r, lat, rop, sc, slots, eps=1e-6, positions=pos, inv_freq=f)
        return kd.latent_cache_read(lat, rop, sc, table, loc, lat.shape[0] * 32)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (3, 4, 5):
        x.copy_(normal(200, 512, seed=seed, dtype=BF16))
        start = r.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        r.copy_(start)
        assert torch.equal(both(), got)


def test_empty():
    lat, rop, _ = (None if t is None else t.cuda() for t in ref.cache(2, 4, 64, 8, BF16))
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    kd.latent_cache_write(lat[0, :0], rop[0, :0], lat, rop, None, none)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    loc = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert kd.latent_cache_read(lat, rop, None, table, loc, 0).shape == (0, 72)
    x = torch.empty(0, 3, 64, device="cuda")
    assert kd.rotary_embedding(x, none, ref.frequencies(64).cuda()).shape == x.shape
