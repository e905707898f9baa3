"""Rotation, latent cache and attention on the host: status codes of the C entry points (no call
reaches a launch), what the bindings refuse, and the FP64 definitions on examples worked out by
hand."""

import ctypes
import math

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd
from packed_varlen_causal_depthwise_amd import _lib
from packed_varlen_causal_depthwise_amd._lib import EINVAL, EUNSUPPORTED, OK

A = 0x10000  # an aligned address that nothing reads
BIG = 1 << 31


def cache_of(**kw):
    a = dict(latents=A, ropes=A, scales=0, pages=9, page=16, latent=512, rope=64, l0=16 * 512, l1=512,
             r0=16 * 64, r1=64, s0=0, s1=0, dt=_lib.BF16, e4m3=0)
    assert set(kw) <= set(a)
    return _lib.LATENT_CACHE.pack(*{**a, **kw}.values())


BAD_CACHES = [
    (dict(pages=-1), EINVAL), (dict(page=0), EINVAL), (dict(latent=0), EINVAL), (dict(rope=-8), EINVAL),
    (dict(dt=3), EINVAL), (dict(dt=_lib.F32), EUNSUPPORTED), (dict(latent=516), EUNSUPPORTED),
    (dict(latent=520, l0=16 * 520, l1=520), EUNSUPPORTED), (dict(rope=72, r0=16 * 72, r1=72), EUNSUPPORTED),
    (dict(rope=4), EUNSUPPORTED), (dict(pages=BIG), EUNSUPPORTED), (dict(page=BIG), EUNSUPPORTED),
    (dict(pages=1 << 16, page=1 << 15), EUNSUPPORTED), (dict(l0=-8), EUNSUPPORTED), (dict(l1=513), EUNSUPPORTED),
    (dict(r1=68), EUNSUPPORTED), (dict(r0=-1024), EUNSUPPORTED), (dict(latents=0), EINVAL), (dict(ropes=0), EINVAL),
    (dict(latents=A + 8), EUNSUPPORTED), (dict(ropes=A + 2), EUNSUPPORTED),
    (dict(e4m3=1, scales=0), EINVAL), (dict(e4m3=1, scales=A, latent=40), EUNSUPPORTED),
    (dict(e4m3=1, scales=A, l1=520), EUNSUPPORTED), (dict(e4m3=1, scales=A, s0=-1), EUNSUPPORTED),
]


def attend_code(update=0, workspace=A, size=1 << 40, cache=None, **kw):
    a = dict(ql=A, qr=A, table=A, lens=A, loc=0 if update else A, out=A, tokens=5, seqs=5 if update else 2, heads=12,
             ql0=12 * 512, ql1=512, qr0=12 * 64, qr1=64, ts=7, width=7, scale=0.1)
    assert set(kw) <= set(a)
    packed = cache_of(**(cache or {})) + _lib.LATENT_ARGS.pack(*{**a, **kw}.values())
    return _lib.load().kdaconv_latent_attention_validate(packed, update, workspace, size)


@pytest.mark.parametrize("update", [0, 1])
@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(tokens=-1), EINVAL), (dict(heads=-1), EINVAL), (dict(width=-1), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(ql=0), EINVAL), (dict(qr=0), EINVAL), (dict(lens=0), EINVAL), (dict(table=0), EINVAL), (dict(out=0), EINVAL),
    (dict(table=0, width=0), OK), (dict(ql=A + 1), EUNSUPPORTED), (dict(ql=A + 2), OK), (dict(out=A + 1), EUNSUPPORTED),
    (dict(lens=A + 2), EUNSUPPORTED), (dict(table=A + 1), EUNSUPPORTED), (dict(ql0=-1), EUNSUPPORTED),
    (dict(qr1=-64), EUNSUPPORTED), (dict(ts=-7), EUNSUPPORTED), (dict(heads=65536), EUNSUPPORTED),
    (dict(workspace=0), EINVAL), (dict(workspace=A + 16), EUNSUPPORTED), (dict(size=4096), EINVAL),
    (dict(heads=0, ql=0, qr=0, out=0, workspace=0, size=0), OK),
])
def test_attention_codes(update, kw, code):
    assert attend_code(update, **kw) == code


def test_attention_codes_of_either_form():
    assert attend_code(1, tokens=4) == EINVAL  # a token per sequence
    assert attend_code(0, loc=0) == EINVAL
    assert attend_code(0, loc=A + 2) == EUNSUPPORTED
    assert attend_code(0, tokens=1 << 26, heads=64) == EUNSUPPORTED  # 2^32 rows
    assert attend_code(0, seqs=1 << 30) == EUNSUPPORTED
    assert attend_code(0, width=BIG) == EUNSUPPORTED
    assert attend_code(0, qr=0, cache=dict(rope=0)) == OK
    lib = _lib.load()
    assert lib.kdaconv_latent_attention_validate(None, 0, A, 1 << 40) == EINVAL
    assert lib.kdaconv_latent_attention(None, A, 1 << 40, None) == EINVAL


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_codes(kw, code):
    lib, packed = _lib.load(), cache_of(**kw)
    assert attend_code(cache=kw) == code
    assert lib.kdaconv_latent_cache_write(packed, A, 512, A, 64, 3, A, 0, None, -1.0, None, 0, None, 0, 1.0, None) == code
    assert lib.kdaconv_latent_cache_read(packed, A, 7, 7, A, 2, 9, A, None) == code


def test_workspace():
    size = _lib.load().kdaconv_latent_attention_workspace
    assert size(0, 3, 4, 512) == size(3, 0, 4, 512) == size(3, 3, 0, 512) == 0
    # 16, 32 or 64 rows of sums with two more words each, for both ends of 256 parts.
    shared = 256 * 2 * 16
    for tokens, seqs, heads, rows in ((1, 1, 16, 16), (1, 1, 17, 32), (2, 1, 16, 32), (9, 1, 4, 64), (1000, 10, 128, 64)):
        assert size(tokens, seqs, heads, 512) == shared + 2 * 256 * rows * 514 * 4


def expanded_code(workspace=0, size=0, **kw):
    a = dict(q=A, k=A, kr=A, v=A, qsl=A, ksl=A, out=A, tokens=9, keys=20, seqs=2, heads=12, key=128, rope=64, value=128,
             q0=12 * 192, q1=192, k0=12 * 256, k1=256, kr0=64, v0=12 * 256, v1=256, scale=0.1, dt=_lib.F16, causal=1)
    assert set(kw) <= set(a)
    return _lib.load().kdaconv_expanded_attention_validate(
        _lib.EXPANDED_ARGS.pack(*{**a, **kw}.values()), workspace, size)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(tokens=-1), EINVAL), (dict(keys=-1), EINVAL), (dict(seqs=-1), EINVAL), (dict(heads=-1), EINVAL),
    (dict(key=0), EINVAL), (dict(value=0), EINVAL), (dict(rope=-8), EINVAL), (dict(scale=math.nan), EINVAL), (dict(dt=7), EINVAL),
    (dict(dt=_lib.F32), EUNSUPPORTED), (dict(key=132), EUNSUPPORTED), (dict(key=136), EUNSUPPORTED),
    (dict(value=4), EUNSUPPORTED), (dict(rope=72), EUNSUPPORTED), (dict(k0=12 * 256 + 4), EUNSUPPORTED),
    (dict(v1=252), EUNSUPPORTED), (dict(kr0=65), EUNSUPPORTED), (dict(q0=12 * 192 + 1, q1=193), OK),
    (dict(q0=-1), EUNSUPPORTED), (dict(k1=-256), EUNSUPPORTED), (dict(v0=1 << 23), EUNSUPPORTED),
    (dict(heads=65536), EUNSUPPORTED), (dict(tokens=1 << 30), EUNSUPPORTED), (dict(keys=1 << 30), EUNSUPPORTED),
    (dict(seqs=1 << 23), EUNSUPPORTED), (dict(q=0), EINVAL), (dict(out=0), EINVAL), (dict(qsl=0), EINVAL), (dict(ksl=0), EINVAL),
    (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(kr=0), EINVAL), (dict(k=0, v=0, kr=0, keys=0), OK), (dict(kr=0, rope=0, kr0=0), OK),
    (dict(q=A + 1), EUNSUPPORTED), (dict(k=A + 8), EUNSUPPORTED), (dict(v=A + 2), EUNSUPPORTED), (dict(kr=A + 8), EUNSUPPORTED),
    (dict(ksl=A + 1), EUNSUPPORTED), (dict(tokens=0, q=0, k=0, v=0, out=0), OK),
])
def test_expanded_codes(kw, code):
    assert expanded_code(**kw) == code


def test_expanded_null():
    lib = _lib.load()
    assert lib.kdaconv_expanded_attention_validate(None, A, 1 << 40) == EINVAL
    assert lib.kdaconv_expanded_attention(None, A, 1 << 40, None) == EINVAL


def test_expanded_workspace():
    size = _lib.load().kdaconv_expanded_attention_workspace
    assert size(9, 20, 2, 12, 128) == size(0, 9999, 1, 1, 8) == size(1, 0, 1, 1, 8) == size(1, 9999, 0, 1, 8) == 0
    # Blocks of 128 rows, 2 sequences of 3 heads, at most 256 / 6 parts of 4 steps of 64 keys.
    assert size(9, 2 * 64 * 4 * 2, 2, 3, 40) == 2 * 3 * 2 * 128 * 42 * 4
    assert size(9, 1 << 20, 2, 3, 40) == 2 * 3 * 42 * 128 * 42 * 4
    assert size(9, 1 << 20, 2, 65, 40) == 0 and size(9, 2 * 64 * 8 - 1, 2, 3, 40) == 0
    assert size(600, 4095, 2, 3, 40) == 6 * 3 * 7 * 128 * 42 * 4
    # Of 256 rows over 2048 keys or more.
    assert size(600, 4096, 2, 3, 40) == 4 * 3 * 8 * 256 * 42 * 4
    assert size(2000, 1 << 16, 1, 16, 40) == 8 * 16 * 2 * 256 * 42 * 4
    assert size(2000, 1 << 16, 1, 17, 40) == 0
    kw = dict(keys=2048, seqs=2)
    assert expanded_code(**kw) == EINVAL and expanded_code(A, 1 << 30, **kw) == OK
    assert expanded_code(A + 16, 1 << 30, **kw) == EUNSUPPORTED and expanded_code(A, 9999, **kw) == EINVAL


def rotary_code(**kw):
    a = dict(x=A, dt=_lib.BF16, tokens=3, heads=2, dim=192, x0=384, x1=192, pos=A, wide=0, freq=A, rotary=64, offset=128,
             inter=0, scale=1.0, out=A, o0=384, o1=192, stream=None)
    assert set(kw) <= set(a)
    return _lib.load().kdaconv_rotary_embedding(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), OK), (dict(heads=0), OK), (dict(tokens=-1), EINVAL), (dict(heads=-1), EINVAL), (dict(dim=0), EINVAL),
    (dict(dt=9), EINVAL), (dict(rotary=0), EINVAL), (dict(rotary=63), EINVAL), (dict(offset=-1), EINVAL), (dict(offset=129), EINVAL),
    (dict(rotary=194, offset=0), EINVAL), (dict(x0=-1), EUNSUPPORTED), (dict(o1=-192), EUNSUPPORTED), (dict(o1=191), EINVAL),
    (dict(o0=191), EINVAL), (dict(x=0), EINVAL), (dict(out=0), EINVAL), (dict(pos=0), EINVAL), (dict(freq=0), EINVAL),
    (dict(x=A + 1), EUNSUPPORTED), (dict(dt=_lib.F32, x=A + 2), EUNSUPPORTED), (dict(pos=A + 2), EUNSUPPORTED),
    (dict(wide=1, pos=A + 4), EUNSUPPORTED), (dict(freq=A + 2), EUNSUPPORTED), (dict(tokens=1 << 31), EUNSUPPORTED),
    (dict(heads=1 << 16), EUNSUPPORTED), (dict(dim=1 << 17, x1=1 << 17, o1=1 << 17, o0=1 << 18), EUNSUPPORTED),
    (dict(dim=40000, rotary=40000, offset=0, x1=40000, o1=40000, o0=80000), EUNSUPPORTED),
])
def test_rotary_codes(kw, code):
    assert rotary_code(**kw) == code


def write_code(cache=None, **kw):
    a = dict(latent=A, ls=512, rope=A, rs=64, tokens=3, slots=A, wide=0, weight=None, eps=1e-6, pos=A, far=0, freq=A, inter=0,
             scale=1.0, stream=None)
    assert set(kw) <= set(a)
    return _lib.load().kdaconv_latent_cache_write(cache_of(**(cache or {})), *{**a, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0, latent=None, rope=None, slots=None), OK), (dict(cache=dict(pages=0)), OK), (dict(tokens=-1), EINVAL),
    (dict(eps=math.nan), EINVAL), (dict(tokens=1 << 31), EUNSUPPORTED), (dict(ls=-1), EUNSUPPORTED), (dict(rs=-1), EUNSUPPORTED),
    (dict(latent=None), EINVAL), (dict(rope=None), EINVAL), (dict(slots=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(latent=A + 1), EUNSUPPORTED), (dict(slots=A + 2), EUNSUPPORTED), (dict(wide=1, slots=A + 4), EUNSUPPORTED),
    (dict(weight=A + 2), EUNSUPPORTED), (dict(cache=dict(l1=0)), EINVAL), (dict(cache=dict(r1=32)), EINVAL),  # places overlap
    (dict(cache=dict(l0=256, l1=512)), EINVAL),
])
def test_write_codes(kw, code):
    assert write_code(**kw) == code


@pytest.mark.parametrize("args,code", [
    ((A, 7, 7, A, 0, 9, A), OK), ((A, 7, 7, A, 2, 0, A), OK), ((A, 7, 7, A, 2, -1, A), EINVAL), ((A, 7, 7, A, -2, 9, A), EINVAL),
    ((A, 7, -1, A, 2, 9, A), EINVAL), ((A, -7, 7, A, 2, 9, A), EUNSUPPORTED), ((A, 7, 7, None, 2, 9, A), EINVAL),
    ((A, 7, 7, A, 2, 9, None), EINVAL), ((None, 7, 7, A, 2, 9, A), EINVAL), ((A + 2, 7, 7, A, 2, 9, A), EUNSUPPORTED),
    ((A, 7, 7, A + 2, 2, 9, A), EUNSUPPORTED), ((A, 7, 7, A, 2, 9, A + 8), EUNSUPPORTED), ((A, 7, 7, A, 2, BIG, A), EUNSUPPORTED),
    ((A, 7, BIG, A, 2, 9, A), EUNSUPPORTED),
])
def test_read_codes(args, code):
    assert _lib.load().kdaconv_latent_cache_read(cache_of(), *args, None) == code


# The bindings, with tensors on the CPU: the last refusal of each is that.

BF = torch.bfloat16
I32 = torch.int32


def refuses(f, args, kw, changes):
    for change, match in changes:
        a, k = list(args), dict(kw)
        for key, value in change.items():
            if isinstance(key, int):
                a[key] = value
            else:
                k[key] = value
        with pytest.raises(ValueError, match=match):
            f(*a, **k)


def test_rotary_refuses():
    x, pos, freq = torch.zeros(3, 2, 24, dtype=BF), torch.zeros(3, dtype=I32), torch.zeros(4)
    refuses(kd.rotary_embedding, (x, pos, freq), {}, [
        ({0: x[0]}, "tokens, heads, head_dim"), ({0: x.double()}, "float32"), ({0: x.transpose(1, 2)}, "contiguous"),
        ({1: pos[:2]}, "positions must"), ({1: pos.float()}, "positions must"), ({2: freq.double()}, "inv_freq must"),
        ({2: freq[None]}, "inv_freq must"), (dict(out=x.half()), "out must"), (dict(out=x[:2]), "out must"), ({}, "GPU tensor")])
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, factor=0.5),
               dict(rotary_dim=8, original_length=0), dict(rotary_dim=8, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            kd.rotary_frequencies(device="cpu", **kw)


def cache_tensors(dtype=BF, e4m3=False):
    return list(ref.cache(4, 8, 64, 16, dtype, e4m3))


BAD_TENSORS = [
    (lambda c: c.__setitem__(0, c[0][0]), "latents must be"), (lambda c: c.__setitem__(1, c[1][:3]), "latents must be"),
    (lambda c: c.__setitem__(1, c[1].float()), "bfloat16 or float16"), (lambda c: c.__setitem__(0, c[0].half()), "dtype of ropes"),
    (lambda c: c.__setitem__(0, c[0].transpose(1, 2).contiguous().transpose(1, 2)), "last axis"),
    (lambda c: c.__setitem__(2, torch.zeros(4, 8, 2, dtype=torch.uint8)), "scales belong"),
    (lambda c: c.__setitem__(0, c[0].to(torch.float8_e4m3fn)), "need uint8 scales"),
    (lambda c: (c.__setitem__(0, c[0].to(torch.float8_e4m3fn)), c.__setitem__(2, torch.zeros(4, 8, 3, dtype=torch.uint8))),
     "need uint8 scales"),
]


@pytest.mark.parametrize("change,match", BAD_TENSORS)
def test_cache_tensors_refused(change, match):
    c = cache_tensors()
    change(c)
    with pytest.raises(ValueError, match=match):
        kd.latent_cache_write(torch.zeros(3, 64, dtype=BF), torch.zeros(3, 16, dtype=BF), *c, torch.zeros(3, dtype=I32))
    with pytest.raises(ValueError, match=match):
        kd.latent_cache_read(*c, torch.zeros(1, 2, dtype=I32), torch.tensor([0, 5], dtype=I32), 5)
    with pytest.raises(ValueError, match=match):
        kd.latent_attention_update(torch.zeros(1, 2, 64, dtype=BF), torch.zeros(1, 2, 16, dtype=BF), *c,
                                   torch.zeros(1, 2, dtype=I32), torch.ones(1, dtype=I32), scale=1.0)


def test_write_refuses():
    c, slots = cache_tensors(), torch.zeros(3, dtype=torch.int64)
    x, r = torch.zeros(3, 64, dtype=BF), torch.zeros(3, 16, dtype=BF)
    freq = torch.zeros(8)
    refuses(kd.latent_cache_write, (x, r, *c, slots), {}, [
        ({0: x[:, :32]}, "latent must be"), ({1: r[:2]}, "latent must be"), ({0: x.half()}, "dtype of ropes"),
        ({0: torch.zeros(64, 3, dtype=BF).t()}, "columns"), ({5: slots[:2]}, "slots must"), ({5: slots.double()}, "slots must"),
        (dict(weight=torch.zeros(64)), "give eps"), (dict(eps=-1.0), "negative"), (dict(eps=math.nan), "negative"),
        (dict(eps=1e-6, weight=torch.zeros(63)), "weight must"), (dict(eps=1e-6, weight=torch.zeros(64, dtype=BF)), "weight must"),
        (dict(inv_freq=freq[:4]), "rope_dim / 2"), (dict(inv_freq=freq), "needs positions"),
        (dict(inv_freq=freq, positions=slots[:2]), "positions must"), ({}, "GPU tensor")])


def test_read_refuses():
    c = cache_tensors(e4m3=True)
    table, loc = torch.zeros(2, 3, dtype=I32), torch.tensor([0, 4, 9], dtype=I32)
    refuses(kd.latent_cache_read, (*c, table, loc, 9), {}, [
        ({3: table.long()}, "block_table must"), ({3: table[:1]}, "block_table must"), ({3: table[0]}, "block_table must"),
        ({3: torch.zeros(3, 2, dtype=I32).t()}, "columns"), ({4: loc.long()}, "kv_start_loc"), ({4: loc[None]}, "kv_start_loc"),
        (dict(out=torch.zeros(9, 80)), "out must"), (dict(out=torch.zeros(8, 80, dtype=BF)), "out must"), ({}, "GPU tensor")])


def test_attention_refuses():
    c, table, lens = cache_tensors(), torch.zeros(3, 2, dtype=I32), torch.ones(3, dtype=I32)
    q, r, loc = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, 2, 16, dtype=BF), torch.tensor([0, 1, 2, 3], dtype=I32)
    changes = [
        ({0: q[:, :, :32]}, "q_latent must"), ({1: r[:, :1]}, "q_latent must"), ({0: q.half()}, "dtype of ropes"),
        ({0: torch.zeros(3, 64, 2, dtype=BF).transpose(1, 2)}, "last axis"), ({5: table[:2]}, "block_table"),
        ({6: lens[:2]}, "seq_lens"), ({6: lens.long()}, "seq_lens"), ({6: torch.ones(6, dtype=I32)[::2]}, "seq_lens"),
        (dict(out=q.half()), "out must"), ({}, "GPU tensor")]
    refuses(kd.latent_attention_update, (q, r, *c, table, lens), dict(scale=1.0), changes)
    refuses(kd.latent_attention_fn, (q, r, *c, table, lens, loc), dict(scale=1.0), changes)
    refuses(kd.latent_attention_fn, (q, r, *c, table, lens, loc), dict(scale=1.0),
            [({7: loc.long()}, "query_start_loc"), ({7: loc[None]}, "query_start_loc")])
    assert not kd.latent_attention_supported(q, r, *c)  # not on a GPU


def test_expanded_refuses():
    q, k, r, v = (torch.zeros(*s, dtype=BF) for s in ((5, 2, 24), (9, 2, 16), (9, 8), (9, 2, 16)))
    loc = torch.tensor([0, 5], dtype=I32)
    refuses(kd.expanded_attention_fn, (q, k, r, v, loc, torch.tensor([0, 9], dtype=I32)), {}, [
        ({0: q[0]}, "q must be"), ({1: k[:8]}, "q must be"), ({3: v[:, :1]}, "q must be"), ({2: r[:8]}, "k_rope must"),
        ({2: None}, "channels"), ({0: q[:, :, :16]}, "channels"), ({0: q.half()}, "one dtype"), ({2: r.half()}, "one dtype"),
        ({0: torch.zeros(5, 24, 2, dtype=BF).transpose(1, 2)}, "last axis"), ({4: loc.long()}, "query_start_loc"),
        ({5: torch.zeros(3, dtype=I32)}, "as many entries"), (dict(out=torch.zeros(5, 2, 16)), "out must"), ({}, "GPU tensor")])
    assert not kd.expanded_attention_supported(q, k, r, v)


def test_frequencies():
    f, m = kd.rotary_frequencies(8, 10000.0, device="cpu")
    assert torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001])) and m == 1.0
    f, m = kd.rotary_frequencies(64, factor=32.0, original_length=4096, device="cpu")
    plain, _ = kd.rotary_frequencies(64, device="cpu")
    # Pairs below 32 turns in 4096 positions: 10000^(-i/32) * 4096 / (2 pi) = 32 at i = 10.47, 1 turn at i = 22.5.
    assert torch.equal(f[:11], plain[:11]) and torch.equal(f[23:], (plain.double() / 32).float()[23:])
    assert bool(((f[11:23] < plain[11:23]) & (f[11:23] > plain[11:23] / 32)).all())
    assert m == 0.1 * math.log(32.0) + 1


def test_definitions_by_hand():
    """Two cached tokens, latents (1, 0, ..) and (3, 0, ..), scores 0 and ln 3: weights 1/4 and
    3/4, the sum 2.5; and rounding to 8 bits."""
    latents, ropes = torch.zeros(1, 2, 8, dtype=torch.float64), torch.zeros(1, 2, 2, dtype=torch.float64)
    latents[0, :, 0] = torch.tensor([1.0, 3.0])
    ropes[0, 1, 1] = math.log(3.0)
    q, r = torch.zeros(2, 1, 8), torch.zeros(2, 1, 2, dtype=torch.float64)
    r[:, 0, 1] = 2.0
    out = ref.attention(q, r, latents, ropes, None, torch.tensor([[0]]), [2], [0, 2], 0.5)
    assert abs(out[1, 0, 0] - 2.5) < 1e-12 and out[0, 0, 0] == 1.0  # token 0 does not see token 1
    e = ref.expanded(torch.cat((q, r), -1), latents[0][:, None], ropes[0], latents[0][:, None], [0, 2], [0, 2], 0.5)
    assert torch.allclose(e, out, atol=1e-12)
    assert ref.attention(q, r, latents, ropes, None, torch.tensor([[7]]), [2], [0, 2], 0.5).abs().max() == 0
    y = torch.zeros(32)
    y[:5] = torch.tensor([449.0, -2.125, 1.0, math.inf, 0.0])
    v, s = ref.to_8_bits(y)
    # 449 needs 2^1: 224.5 rounds to 224 in steps of 16, -1.0625 halfway to the even -1.
    assert s.item() == 128 and v[:3].tolist() == [224.0, -1.0, 0.5] and bool(v[3].isnan()) and v[4] == 0
    x = ref.turned(torch.tensor([[[1.0, 0.0, 5.0, 7.0]]]), torch.tensor([1]), torch.tensor([math.pi / 2, 0.0]), False)
    assert torch.allclose(x, torch.tensor([[[-5.0, 0.0, 1.0, 7.0]]]).double(), atol=1e-6)


def test_packed_sizes_match_the_header():
    """Structs of 8-byte members, doubles and a pair of ints, without padding."""
    assert _lib.LATENT_CACHE.size == 3 * 8 + 10 * 8 + 2 * 4 and _lib.LATENT_CACHE.size % 8 == 0
    assert _lib.LATENT_ARGS.size == 6 * 8 + 9 * 8 + 8 and _lib.EXPANDED_ARGS.size == 7 * 8 + 14 * 8 + 8 + 8
    assert ctypes.sizeof(ctypes.c_void_p) == 8
