"""Refusals of the gated delta rule and the norms, on the host: the C checks (no HIP call)
and the binding's."""

import pytest
import torch

import packed_varlen_causal_depthwise_amd as kd
import rule_reference as ref
from packed_varlen_causal_depthwise_amd import _lib

A = 0x10000  # an aligned address that is never followed

FIELDS = ("q k v g beta a_log dt_bias states qsl ci init out T S H HK D qs0 qs1 ks0 ks1 vs0 vs1 gs0 "
          "gs1 gs2 bs0 bs1 lines ss0 ss1 cis null scale l2 lower dt gdt bdt gate logits has_null").split()


def pack(**kw):
    a = dict.fromkeys("q k v g beta a_log dt_bias states qsl ci init out".split(), A)
    a.update(T=100, S=3, H=4, HK=2, D=128, qs0=256, qs1=128, ks0=256, ks1=128, vs0=512, vs1=128,
             gs0=512, gs1=128, gs2=1, bs0=4, bs1=1, lines=9, ss0=65536, ss1=16384, cis=1, null=0,
             scale=0.1, l2=1e-6, lower=-5.0, dt=_lib.BF16, gdt=_lib.BF16, bdt=_lib.F32,
             gate=_lib.GATE_BOUNDED, logits=1, has_null=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return _lib.RULE_ARGS.pack(*(a[f] for f in FIELDS))


OK, EINVAL, EUNSUPPORTED = _lib.OK, _lib.EINVAL, _lib.EUNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    ({}, OK),
    (dict(T=-1), EINVAL), (dict(S=-1), EINVAL), (dict(H=-1), EINVAL), (dict(lines=-1), EINVAL),
    (dict(HK=0), EINVAL), (dict(HK=3), EINVAL), (dict(D=0), EINVAL),
    (dict(dt=7), EINVAL), (dict(gdt=-1), EINVAL), (dict(bdt=3), EINVAL), (dict(gate=3), EINVAL),
    (dict(gs2=2), EINVAL), (dict(gs2=0), OK),
    (dict(lower=0.5), EINVAL), (dict(lower=float("nan")), EINVAL), (dict(lower=0.0), OK),
    (dict(D=96), EUNSUPPORTED), (dict(D=256), EUNSUPPORTED), (dict(D=64), OK),
    (dict(gdt=_lib.F16), EUNSUPPORTED), (dict(bdt=_lib.F16), EUNSUPPORTED),
    (dict(dt=_lib.F32, gdt=_lib.BF16), EUNSUPPORTED), (dict(gdt=_lib.F32), OK),
    (dict(qs0=-1), EUNSUPPORTED), (dict(vs0=1 << 24), EUNSUPPORTED), (dict(bs1=-4), EUNSUPPORTED),
    (dict(ss0=-1), EUNSUPPORTED), (dict(cis=-1), EUNSUPPORTED),
    (dict(T=1 << 31), EUNSUPPORTED), (dict(H=70000, HK=1), EUNSUPPORTED),
    (dict(q=0), EINVAL), (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(g=0), EINVAL),
    (dict(beta=0), EINVAL), (dict(states=0), EINVAL), (dict(ci=0), EINVAL), (dict(out=0), EINVAL),
    (dict(a_log=0), EINVAL), (dict(a_log=0, gate=_lib.GATE_LOG), OK), (dict(dt_bias=0), OK),
    (dict(init=0), OK),
    (dict(q=A + 1), EUNSUPPORTED), (dict(q=A + 2), OK), (dict(out=A + 1), EUNSUPPORTED),
    (dict(states=A + 2), EUNSUPPORTED), (dict(beta=A + 2), EUNSUPPORTED),
    (dict(T=0, S=0, q=0, out=0), OK),
])
def test_status_codes(kw, code):
    lib = _lib.load()
    update = dict(S=100)
    update.update(kw)
    if "S" not in kw and "T" in kw:
        update["S"] = kw["T"]
    assert lib.kdaconv_gated_delta_rule_validate(pack(**update), 1, None, 0) == code
    # the prefill: the same, with scratch memory as large as any size needs
    assert lib.kdaconv_gated_delta_rule_validate(pack(**kw), 0, A, 1 << 50) == code


def test_prefill_and_update_checks():
    lib = _lib.load()
    assert lib.kdaconv_gated_delta_rule_validate(None, 0, None, 0) == EINVAL
    assert lib.kdaconv_gated_delta_rule_validate(pack(qsl=0), 0, A, 1 << 50) == EINVAL
    assert lib.kdaconv_gated_delta_rule_validate(pack(S=100, qsl=0), 1, None, 0) == OK
    assert lib.kdaconv_gated_delta_rule_validate(pack(S=99), 1, None, 0) == EINVAL
    need = lib.kdaconv_gated_delta_rule_workspace(100, 3, 4, 128)
    if need > 0:
        assert lib.kdaconv_gated_delta_rule_validate(pack(), 0, None, need) == EINVAL
        assert lib.kdaconv_gated_delta_rule_validate(pack(), 0, A, need - 1) == EINVAL
        assert lib.kdaconv_gated_delta_rule_validate(pack(), 0, A + 16, need) == EUNSUPPORTED
        assert lib.kdaconv_gated_delta_rule_validate(pack(), 0, A, need) == OK
    # refused before anything is launched
    assert lib.kdaconv_gated_delta_rule(pack(D=96), A, 1 << 50, None) == EUNSUPPORTED
    assert lib.kdaconv_gated_delta_rule_update(pack(S=100, HK=3), None) == EINVAL
    assert lib.kdaconv_gated_delta_rule(pack(T=0), None, 0, None) == OK
    assert lib.kdaconv_gated_delta_rule_update(pack(T=0, S=0), None) == OK


def test_norm_status_codes():
    lib = _lib.load()

    def gated(x=A, dt=_lib.BF16, T=5, H=2, dim=128, xs0=256, xs1=128, z=A, zs0=256, zs1=128, act=1,
              w=A, eps=1e-5, out=A):
        return lib.kdaconv_gated_rms_norm(x, dt, T, H, dim, xs0, xs1, z, zs0, zs1, act, w, eps, out, None)

    assert gated(T=0) == OK and gated(H=0, x=0) == OK
    for kw, code in ((dict(T=-1), EINVAL), (dict(H=-1), EINVAL), (dict(dim=0), EINVAL),
                     (dict(dt=4), EINVAL), (dict(act=3), EINVAL), (dict(eps=-1.0), EINVAL),
                     (dict(eps=float("nan")), EINVAL), (dict(dim=100), EUNSUPPORTED),
                     (dict(dim=520), EUNSUPPORTED), (dict(xs0=-1), EUNSUPPORTED),
                     (dict(T=1 << 30, H=4), EUNSUPPORTED), (dict(x=0), EINVAL), (dict(z=0), EINVAL),
                     (dict(out=0), EINVAL), (dict(x=A + 1), EUNSUPPORTED), (dict(w=A + 2), EUNSUPPORTED)):
        assert gated(**kw) == code, kw

    def residual(x=A, dt=_lib.BF16, T=5, N=256, xs=256, r=A, rs=256, scale=1.0, w=A, eps=1e-5, out=A):
        return lib.kdaconv_residual_rms_norm(x, dt, T, N, xs, r, rs, scale, w, eps, out, None)

    assert residual(T=0) == OK
    for kw, code in ((dict(T=-1), EINVAL), (dict(N=0), EINVAL), (dict(dt=3), EINVAL),
                     (dict(eps=-1.0), EINVAL), (dict(N=16385, rs=16385), EUNSUPPORTED),
                     (dict(xs=-1), EUNSUPPORTED), (dict(rs=255), EINVAL), (dict(x=0), EINVAL),
                     (dict(out=0), EINVAL), (dict(r=A + 1), EUNSUPPORTED), (dict(out=A + 1), EUNSUPPORTED)):
        assert residual(**kw) == code, kw


def bad(change, match, update=False):
    args, kw = ref.rule_inputs([4, 3] if not update else [1] * 7, heads=2, qk_heads=1)
    change(args, kw)
    with pytest.raises(ValueError, match=match):
        if update:
            kd.gated_delta_rule_update(*args[:6], args[7], **kw)
        else:
            kd.gated_delta_rule_fn(*args, **kw)


@pytest.mark.parametrize("i,value,match", [
    (0, torch.zeros(7, 128), "q and k"),
    (1, torch.zeros(7, 2, 128, dtype=torch.bfloat16), "q and k"),
    (2, torch.zeros(6, 2, 128, dtype=torch.bfloat16), "agree"),
    (2, torch.zeros(7, 2, 128), "one dtype"),
    (3, torch.zeros(7, 2, 64, dtype=torch.bfloat16), "g must"),
    (3, torch.zeros(7, 2, 128, dtype=torch.float16), "g and beta"),
    (4, torch.zeros(7, 3, dtype=torch.bfloat16), "beta must"),
    (5, torch.zeros(4, 2, 128, 64), "states must"),
    (5, torch.zeros(4, 2, 128, 128, dtype=torch.bfloat16), "states must"),
    (5, torch.zeros(4, 2, 128, 128).transpose(2, 3), "last two axes"),
    (7, torch.zeros(2, dtype=torch.int64), "cache_indices"),
    (7, torch.zeros(1, dtype=torch.int32), "cache_indices"),
])
def test_binding_refuses(i, value, match):
    bad(lambda a, kw: a.__setitem__(i, value), match)
    if i != 7 or value.dtype != torch.int32:
        bad(lambda a, kw: a.__setitem__(i, value), match, update=True)


def test_binding_refuses_more():
    bad(lambda a, kw: None, "GPU tensor")
    bad(lambda a, kw: None, "GPU tensor", update=True)
    bad(lambda a, kw: a.__setitem__(6, a[6].long()), "query_start_loc")
    bad(lambda a, kw: a.__setitem__(8, torch.zeros(1, dtype=torch.bool)), "has_initial_state")
    bad(lambda a, kw: a.__setitem__(8, torch.zeros(2)), "has_initial_state")
    bad(lambda a, kw: kw.update(a_log=None), "need a_log")
    bad(lambda a, kw: kw.update(a_log=torch.zeros(3)), "a_log must")
    bad(lambda a, kw: kw.update(dt_bias=torch.zeros(2, 64)), "dt_bias must")
    bad(lambda a, kw: kw.update(lower_bound=1.0), "lower_bound")
    bad(lambda a, kw: kw.update(out=torch.zeros(7, 2, 128)), "out must")
    bad(lambda a, kw: a.__setitem__(2, torch.zeros(7, 128, 2, dtype=torch.bfloat16).transpose(1, 2)),
        "last axis")
    assert not kd.gated_delta_rule_supported(*ref.rule_inputs([4])[0][:6])  # not on a GPU


def test_norm_binding_refuses():
    x = torch.zeros(3, 2, 64)
    for args, kw, match in (
            ((x[0], None, None), {}, "tokens, heads, dim"), ((x.double(), None, None), {}, "float32"),
            ((x, x[:2], None), {}, "gate must"), ((x, x.half(), None), {}, "gate must"),
            ((x, x, torch.zeros(63)), {}, "weight must"), ((x, x, None), dict(activation="gelu"), "activation"),
            ((x, x, None), dict(out=x.half()), "out must"), ((x, x, None), {}, "GPU tensor"),
            ((x.transpose(1, 2), None, None), {}, "contiguous")):
        with pytest.raises(ValueError, match=match):
            kd.gated_rms_norm(*args, **kw)
    y = torch.zeros(3, 64)
    for args, kw, match in (
            ((x, None, None), {}, "tokens, hidden"), ((y, y.half(), None), {}, "residual must"),
            ((y, y[:2], None), {}, "residual must"), ((y, y, torch.zeros(64).half()), {}, "weight must"),
            ((y.t(), None, None), {}, "contiguous"), ((y, y, None), {}, "GPU tensor"),
            ((y, y, None), dict(out=torch.zeros(3, 65)), "out must")):
        with pytest.raises(ValueError, match=match):
            kd.residual_rms_norm(*args, **kw)


def test_definition_by_hand():
    """The FP64 definition on a two-token example worked out by hand (one key and one value
    channel count; the others are zero)."""
    q = torch.zeros(2, 1, 64)
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    q[:, 0, 0] = torch.tensor([2.0, 3.0])
    k[:, 0, 0] = torch.tensor([0.5, 1.0])
    v[:, 0, 0] = torch.tensor([4.0, 1.0])
    g = torch.zeros(2, 1, 64)
    g[1] = torch.log(torch.tensor(0.25))
    beta = torch.tensor([[1.0], [0.5]])
    states = torch.zeros(1, 1, 64, 64)
    states[0, 0, 0, 0] = 1.0
    out, st = ref.delta_rule(q, k, v, g, beta, states, torch.tensor([0, 2]), torch.tensor([0]),
                             torch.tensor([True]), qk_l2norm=False, scale=1.0)
    # token 0: S' = 1, u = 4 - 0.5 = 3.5, S = 1 + 0.5 * 3.5 = 2.75, out = 5.5
    # token 1: S' = 0.6875, u = 0.5 (1 - 0.6875) = 0.15625, S = 0.84375, out = 2.53125
    assert out[0, 0, 0] == 5.5 and abs(out[1, 0, 0] - 2.53125) < 1e-7
    assert abs(st[0, 0, 0, 0] - 0.84375) < 1e-7
