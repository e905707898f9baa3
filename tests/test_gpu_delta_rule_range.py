"""The gated delta rule over the whole range of its arguments."""

import pytest
import torch

import packed_varlen_causal_depthwise_amd as kd
import rule_reference as ref
from test_gpu_delta_rule import compare, run

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# Lengths, heads and head_dim: heads of 64; of 128 with 8 waves per chunk; with 4.
FORMS = [([100, 40], 3, 64), ([100, 40], 3, 128), ([1100], 16, 128)]
forms = pytest.mark.parametrize("lengths,heads,dim", FORMS, ids=str)


def log_inputs(lengths, heads, dim, seed=0, **kw):
    return ref.rule_inputs(lengths, heads=heads, dim=dim, dtype=F32, gate="log", seed=seed, **kw)


@forms
@pytest.mark.parametrize("rate", [5.0, 5.5, 6.0, 7.0, 8.5])
def test_uniform_strong_decays(rate, lengths, heads, dim):
    """Decays that 8 tokens of a chunk can hold in one factor and 16 cannot: in every
    channel, then in two of three of one head."""
    args, kw = log_inputs(lengths, heads, dim, seed=60)
    args[3] = torch.full_like(args[3], -rate)
    compare(args, kw)
    args[3][:, 1:] = -0.01
    args[3][:, 0, 1::3] = -0.01
    compare(args, kw)


@forms
@pytest.mark.parametrize("step", [1, 4, 1000])
def test_two_strong_decays_in_a_chunk(step, lengths, heads, dim):
    """Tokens between them meet without either: in every channel, every fourth, one."""
    args, kw = log_inputs(lengths, heads, dim, seed=61)
    args[3] = torch.zeros_like(args[3])
    for at in (10, 20):
        args[3][at::32, :, 2::step] = -60.0
    compare(args, kw)


@forms
@pytest.mark.parametrize("lower_bound", [-6.0, -7.0, -8.0, None])
def test_strong_gates(lower_bound, lengths, heads, dim):
    """The gates at a_log = log 16, their inputs of standard deviation 2."""
    args, kw = ref.rule_inputs(lengths, heads=heads, dim=dim, dtype=F32, seed=62,
                               gate="softplus" if lower_bound is None else "bounded")
    kw["a_log"] = torch.full_like(kw["a_log"], 2.772588722239781)
    kw["lower_bound"] = lower_bound
    args[3] = 2 * args[3]
    compare(args, kw)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seed", range(8))
def test_reflections_beside_a_reset_channel(seed, dim):
    """Equal keys and steps of 2, whose errors grow with the tokens, while a channel without
    any key is reset in every chunk."""
    args, kw = log_inputs([97], 1, dim, seed=70 + seed, logits=False)
    key = args[1][:1].clone()
    key[..., 5] = 0.0
    args[1] = key.expand_as(args[1]).contiguous()
    args[4] = 2 * torch.ones_like(args[4])
    args[3] = torch.zeros_like(args[3])
    args[3][3::32, :, 5] = -300.0
    compare(args, kw)


@forms
def test_weak_decays_beside_a_strong_one(lengths, heads, dim):
    """A strong decay at the third token of every 16: the rows after it, on the side of the
    block's middle, meet by sums that do not carry it, exact to a few 2^-24, and so outputs and
    states to a few times 2^-22, the products' pairs: 2^-20 of the largest. Sums that carry
    it, about 100, are rounded to 2^-17, and so are their differences."""
    args, kw = log_inputs(lengths, heads, dim, seed=80)
    args[3] = torch.full_like(args[3], -0.0123)
    place = torch.cat([torch.arange(n) % 16 for n in lengths])
    args[3][place == 3] = -69.0
    out, st, want, want_st = run(args, kw)
    for got, exact in ((out.cpu()[place >= 3], want[place >= 3]), (st.cpu(), want_st)):
        assert (got.double() - exact).abs().max() <= 2.0 ** -20 * exact.abs().max()


# A state from nothing, in one chunk and over several, token by token, and in segments.
SIZES = [([40, 200, 3], 64), ([40, 200, 3], 128), ([700], 128)]


@pytest.mark.parametrize("lengths,dim", SIZES, ids=str)
@pytest.mark.parametrize("beta", [1e-2, 1e-3, 1e-4, 1e-6, 1e-10])
def test_small_steps(beta, lengths, dim):
    """Updates far below the values that they come from."""
    args, kw = log_inputs(lengths, 2, dim, seed=90, logits=False,
                          initial=torch.zeros(len(lengths), dtype=torch.bool))
    args[4] = args[4] * beta
    compare(args, kw)
    args[4][::7] = 0.0
    args[4][5::50] = 1.0  # and full steps among them
    compare(args, kw)


@pytest.mark.parametrize("lengths,dim", SIZES, ids=str)
@pytest.mark.parametrize("length", [1e-2, 1e-4, 1e-6, 30.0])
def test_keys_of_any_length(length, lengths, dim):
    """Keys as they are, much shorter than 1, and longer."""
    args, kw = log_inputs(lengths, 2, dim, seed=91, logits=False,
                          initial=torch.zeros(len(lengths), dtype=torch.bool))
    args[1] = args[1] / args[1].norm(dim=-1, keepdim=True) * length
    args[4] = args[4] / max(1.0, length * length)
    compare(args, kw, qk_l2norm=False)


@pytest.mark.parametrize("lengths,dim", SIZES, ids=str)
@pytest.mark.parametrize("operand", ["q", "k"])
@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e-8, 1e-20, 1e-30])
def test_short_keys_and_queries(size, operand, lengths, dim):
    """Lengths that vanish beside the normalisation's 1e-6."""
    args, kw = log_inputs(lengths, 2, dim, seed=92,
                          initial=torch.zeros(len(lengths), dtype=torch.bool))
    args["qk".index(operand)] *= size
    compare(args, kw)
    args["qk".index(operand)][1::5] /= size  # and ordinary rows among them
    compare(args, kw)


def shortest(size, operand, dim):
    args, kw = log_inputs([40, 100, 3], 2, dim, seed=93, logits=False)
    args[1] = args[1] / args[1].norm(dim=-1, keepdim=True)
    args["qk".index(operand)] = args["qk".index(operand)] * size
    args["qk".index(operand)][7] = 0.0
    return args, kw


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("operand", ["q", "k"])
@pytest.mark.parametrize("size", [1e-30, 1e-36, 1e-38])
def test_shortest_keys_and_queries_as_they_are(size, operand, dim):
    """Lengths whose inverse FP32 cannot hold."""
    args, kw = shortest(size, operand, dim)
    compare(args, kw, qk_l2norm=False)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("operand", ["q", "k"])
def test_subnormal_keys_and_queries_as_they_are(operand, dim):
    """A length below 2^-118 is taken as 2^-118 with entries of 2^-29 (a pair's last bit over
    16): of a product with a state's column, whose length is below 2^4 here, that leaves errors
    below 2^-118 * 2^-29 * sqrt(dim) * 2^4 < 2^-139."""
    args, kw = shortest(1e-41, operand, dim)
    out, st, want, want_st = run(args, kw, qk_l2norm=False)
    for got, exact in ((out, want), (st, want_st)):
        err = (got.cpu().double() - exact).abs().max()
        assert err <= ref.ARITHMETIC * exact.abs().max() + 2.0 ** -139


def check_finite(got, want, dtype, what):
    """Finite where the definition is, and those values right."""
    got, finite = got.cpu(), torch.isfinite(want)
    differ = (torch.isfinite(got) != finite).sum().item()
    assert differ == 0, f"{what}: {differ} of {finite.numel()} finite in one alone"
    ref.check(torch.where(finite, got, torch.zeros_like(got)),
              torch.where(finite, want, torch.zeros_like(want)), dtype, what)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("steep", [False, True])
@pytest.mark.parametrize("value", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("operand", ["q", "k", "v", "g", "beta", "state"])
def test_values_that_are_not_finite(operand, value, steep, dim):
    """They reach the tokens after them, and none before: a token of its own per head. (A log
    decay of -infinity is a reset, and all stays finite.)"""
    tokens = [0, 5, 13, 14, 21, 31, 32, 45, 63, 64, 74]
    for lengths in ([75, 3], [12, 3]):
        args, kw = log_inputs(lengths, len(tokens), dim, seed=94, logits=False,
                              initial=torch.ones(2, dtype=torch.bool))
        args = [a.contiguous() for a in args]
        if steep:
            args[3][4::9, :, 7] = -200.0
        for h, t in enumerate(tokens):
            t %= lengths[0]
            if operand == "state":
                args[5][int(args[7][0]), h, 3 + h, 2 * h] = float(value)
            elif operand == "beta":
                args[4][t, h] = float(value)
            else:
                args["qkvg".index(operand)][t, h, 3 * h] = float(value)
        out, st, want, want_st = run(args, kw)
        check_finite(out, want, F32, "out")
        check_finite(st, want_st, F32, "states")


@pytest.mark.parametrize("dtype,dim,heads", [(F32, 64, 3), (BF16, 128, 3), (F16, 128, 16)], ids=str)
@pytest.mark.parametrize("operand", ["q", "k", "v", "g", "beta"])
def test_values_that_are_not_finite_in_long_sequences(operand, dtype, dim, heads):
    """Through segments that run side by side, and with gates; the sequence after it is whole."""
    args, kw = ref.rule_inputs([700, 33], heads=heads, dim=dim, dtype=dtype, seed=95)
    which = args["q k v g beta".split().index(operand)] = \
        args["q k v g beta".split().index(operand)].contiguous()
    if operand == "v":
        which[333, 0, 0], which[400, 1, 5] = float("nan"), float("inf")
    else:
        which[333, 0] = float("nan")
    out, st, want, want_st = run(args, kw)
    check_finite(out, want, dtype, "out")
    check_finite(st, want_st, F32, "states")


def test_supported_asks_for_a_prefill():
    """More tokens times heads than an update may have sequences times heads."""
    one = torch.zeros(1, 64, 128, dtype=BF16, device="cuda")
    x, beta = one.expand(131072, 64, 128), one[..., 0].expand(131072, 64)
    states = torch.zeros(1, 64, 128, 128, device="cuda")
    assert kd.gated_delta_rule_supported(x, x, x, x, beta, states)
    assert kd.gated_delta_rule_supported(x[:0], x[:0], x[:0], x[:0], beta[:0], states)
    assert not kd.gated_delta_rule_supported(x, x, x, x.half(), beta, states)
    wide = torch.empty(3 << 24, dtype=BF16, device="cuda").as_strided((3, 64, 128), (1 << 24, 128, 1))
    assert not kd.gated_delta_rule_supported(wide, x[:3], x[:3], x[:3], beta[:3], states)


def test_one_row_of_a_batch_of_one():
    """One token out of (1, tokens, columns): its token stride is the whole batch."""
    args, kw = ref.rule_inputs([1], heads=4, dim=128, seed=98, initial=torch.tensor([True]))
    rows = torch.zeros(1, 4096, 2500, dtype=BF16, device="cuda")
    row = rows[:, 77]
    assert row.stride(0) > 1 << 23
    g = [a.cuda() for a in args]
    for i in range(4):
        g[i] = row[:, 512 * i + 3:512 * i + 515].view(1, 4, 128).copy_(args[i])
    g[4] = row[:, 2100:2104].copy_(args[4])
    gkw = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    want, want_st = ref.delta_rule(*args, **kw)
    for update in (False, True):
        st = args[5].cuda()
        if update:
            out = kd.gated_delta_rule_update(*g[:5], st, g[7], **gkw, null_block_id=None)
        else:
            out = kd.gated_delta_rule_fn(*g[:5], st, *g[6:], **gkw, null_block_id=None)
        ref.check(out, want, BF16, "out")
        ref.check(st, want_st, F32, "states")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("operand", ["q", "k"])
@pytest.mark.parametrize("lengths", [[1, 1, 1], [9, 40]], ids=str)
def test_long_keys_and_queries(lengths, operand, dtype):
    """Squares past FP32's range, token by token and in chunks."""
    args, kw = ref.rule_inputs(lengths, heads=2, dim=128, dtype=dtype, seed=96)
    args["qk".index(operand)] = (args["qk".index(operand)].double() * 1e25).to(dtype)
    compare(args, kw)


@pytest.mark.parametrize("lengths", [[31], [64, 33], [94, 64, 148, 122]], ids=str)
@pytest.mark.parametrize("beta", [0.1, 1e-3, 1e-5])
@pytest.mark.parametrize("most", [3.0, 12.0, 100.0])
def test_small_steps_after_a_state_that_fades(most, beta, lengths):
    """Decays that leave nothing of a state within a chunk, and updates far below what it was."""
    for dim in (64, 128):
        args, kw = log_inputs(lengths, 2, dim, seed=99, logits=False,
                              initial=torch.ones(len(lengths), dtype=torch.bool))
        gen = torch.Generator().manual_seed(7)
        args[3] = -torch.rand(args[3].shape, generator=gen) * most
        args[4] = args[4] * beta
        compare(args, kw)


@pytest.mark.parametrize("logit", [-5.0, -10.0])
def test_many_small_updates_of_a_long_memory(logit):
    """Each about 2^-20 of the state that it is added to, and hardly any decay."""
    args, kw = ref.rule_inputs([900], heads=20, qk_heads=10, dim=128, dtype=F32, seed=50001)
    kw["a_log"] = torch.full_like(kw["a_log"], 2.772588722239781)
    kw["lower_bound"] = -8.0
    args[3] = 0.3 * args[3]
    args[4] = args[4] + logit
    args[1] = args[1] / args[1].norm(dim=-1, keepdim=True) * 0.01
    compare(args, kw, qk_l2norm=False)
