"""The gated delta rule's kernels against its definition in FP64 (rule_reference)."""

import pytest
import torch

import packed_varlen_causal_depthwise_amd as kd
import rule_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def to_gpu(t):
    """The same values, strides and offset on the GPU."""
    if t is None or not isinstance(t, torch.Tensor):
        return t
    base = t._base if t._base is not None else t
    return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset()) if base.is_contiguous() \
        else t.cuda()


def run(args, kw, **more):
    """(out, states) of the prefill call on the GPU, and of the FP64 definition."""
    gargs = [to_gpu(a) for a in args]
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    null = more.pop("null_block_id", None)
    out = torch.full(args[2].shape, -7.0, dtype=args[2].dtype, device="cuda")
    kd.gated_delta_rule_fn(*gargs, **gkw, null_block_id=null, out=out, **more)
    torch.cuda.synchronize()
    want, states = ref.delta_rule(*args, **kw, null_block_id=null, **more)
    return out, gargs[5], want, states


def compare(args, kw, what="", **more):
    out, st, want, want_st = run(args, kw, **more)
    owned = ~torch.isnan(want[:, 0, 0]) if want.shape[1] else torch.zeros(0, dtype=torch.bool)
    ref.check(out.cpu()[owned], want[owned], args[2].dtype, what + " out")
    assert (out.cpu()[~owned] == -7.0).all(), "rows no sequence owns were written"
    ref.check(st, want_st, F32, what + " states")
    before = args[5]
    touched = {int(args[7][s]) for s in range(len(args[6]) - 1)
               if args[6][s + 1] > args[6][s] or not args[8][s]}
    for line in range(len(before)):
        if line not in touched or line == more.get("null_block_id"):
            assert torch.equal(st[line].cpu(), before[line]), f"line {line} was written"


LENGTHS = [[1], [2, 1], [4, 5], [15, 16, 17], [31, 32, 33], [64], [65, 0, 63], [0, 5, 0, 130, 0],
           [300], [257, 1, 3, 96]]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_lengths(lengths, dim):
    args, kw = ref.rule_inputs(lengths, heads=2, dim=dim, seed=len(lengths) + sum(lengths), pad=3)
    compare(args, kw)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gate", ["log", "softplus", "bounded"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_types_and_gates(dtype, gate, dim):
    gd = F32 if gate == "log" else None
    args, kw = ref.rule_inputs([70, 3, 41], heads=3, dim=dim, dtype=dtype, gate=gate, gate_dtype=gd,
                               seed=5)
    compare(args, kw)


@pytest.mark.parametrize("heads,qk_heads", [(1, 1), (4, 2), (6, 1), (12, 12)])
def test_shared_heads(heads, qk_heads):
    args, kw = ref.rule_inputs([90, 37], heads=heads, qk_heads=qk_heads, dim=128, seed=heads)
    compare(args, kw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_strided_unaligned_rows(dtype):
    for dim in (64, 128):
        args, kw = ref.rule_inputs([50, 33], heads=2, dim=dim, dtype=dtype, strided=True, seed=9)
        assert args[0].storage_offset() == 3
        compare(args, kw)


@pytest.mark.parametrize("per_head,beta_dtype,logits,gate", [
    (True, None, True, "softplus"), (True, F32, False, "log"), (False, F32, False, "bounded")])
def test_gate_per_head_and_beta_forms(per_head, beta_dtype, logits, gate):
    args, kw = ref.rule_inputs([66, 20], heads=3, gate=gate, per_head=per_head,
                               beta_dtype=beta_dtype, logits=logits, seed=12)
    compare(args, kw)


def test_no_bias_no_initial_no_norm_and_scale():
    args, kw = ref.rule_inputs([80, 9], heads=2, seed=4, gate="softplus")
    kw["dt_bias"] = None
    args[8] = None
    compare(args, kw, scale=0.5)
    # unit keys, queries of any length, no normalisation in the call
    args, kw = ref.rule_inputs([80, 9], heads=2, seed=4, dtype=F32)
    args[1] = args[1] / args[1].norm(dim=-1, keepdim=True)
    args[0] = args[0] * 50
    compare(args, kw, qk_l2norm=False)


def test_null_block_and_lines_out_of_range():
    args, kw = ref.rule_inputs([40, 70, 2, 35], heads=2, lines=6, seed=3,
                               initial=torch.tensor([True] * 4))
    args[7] = torch.tensor([2, 0, 99, -1], dtype=torch.int32)
    compare(args, kw, null_block_id=0)


@pytest.mark.parametrize("lengths", [[40], [100, 3]], ids=str)
def test_resets_and_strong_decays(lengths):
    """Log decays of -infinity, far below FP32's exp range, and so strong over 8 tokens that
    products of decays leave the range; and no decay at all."""
    for dim in (64, 128):
        args, kw = ref.rule_inputs(lengths, heads=2, dim=dim, gate="log", gate_dtype=F32, seed=21,
                                   initial=torch.ones(len(lengths), dtype=torch.bool))
        g = args[3]
        g[5, :, :] = -float("inf")
        g[11, :, ::3] = -300.0
        g[12:30, 0, 1::4] = -40.0
        g[20:36, 1, 2::5] = -12.0
        g[33] = 0.0
        compare(args, kw)
        args[3] = torch.zeros_like(g)
        compare(args, kw, "no decay")


def test_strong_decays_in_many_chunks():
    """Chunks whose decays leave the range of products, with the smaller workgroups."""
    args, kw = ref.rule_inputs([1200], heads=16, dim=128, gate="log", gate_dtype=F32, seed=22)
    g = args[3]
    g[5::64, :, :] = -float("inf")
    g[12::64, ::2, 1::4] = -40.0
    g[20::64, 1, 2::5] = -12.0
    for t in range(12, 30):
        g[t::64, ::3, ::7] = -15.0
    compare(args, kw)


def test_equal_keys_with_full_steps():
    """All keys equal and beta one: the triangular system at its worst."""
    for dim in (64, 128):
        args, kw = ref.rule_inputs([97], heads=1, dim=dim, dtype=F32, gate="log", logits=False, seed=8)
        args[1] = args[1][:1].expand_as(args[1]).contiguous()
        args[4] = torch.ones_like(args[4])
        args[3] = torch.zeros_like(args[3])
        compare(args, kw)
        args[4] = 2 * torch.ones_like(args[4])  # reflections
        compare(args, kw)


def test_zero_keys_values_and_states():
    args, kw = ref.rule_inputs([50], heads=2, dtype=F32, seed=2)
    args[1][7:20] = 0.0
    args[0][3] = 0.0
    compare(args, kw)
    args[2] = torch.zeros_like(args[2])
    args[5] = torch.zeros_like(args[5])
    out, st, want, _ = run(args, kw)
    assert (out == 0).all() and (st == 0).all() and (want == 0).all()


@pytest.mark.parametrize("v_scale", [1e-30, 1e-12, 1e-4, 1e4, 1e12, 1e30])
def test_magnitudes(v_scale):
    """Values and states of any size, and of very different sizes by column and over time."""
    args, kw = ref.rule_inputs([75, 40], heads=2, dtype=F32, seed=6, v_scale=v_scale)
    compare(args, kw, str(v_scale))
    args, kw = ref.rule_inputs([140], heads=1, dtype=F32, seed=6, gate="log",
                               initial=torch.tensor([True]))
    args[2][64:] *= v_scale  # values change size on the way
    args[2][:, :, ::2] *= 1e-3
    out, st, want, want_st = run(args, kw)
    for part, exact in ((out[:64].cpu(), want[:64]), (out[64:].cpu(), want[64:]),
                        (st.cpu()[int(args[7][0])], want_st[int(args[7][0])])):
        for cols in (slice(0, None, 2), slice(1, None, 2)):
            ref.check(part[..., cols], exact[..., cols], F32, f"columns {cols}")


def test_unused_memory_is_not_read():
    """NaN in rows no sequence owns, in lines that are not read, and after the last row."""
    args, kw = ref.rule_inputs([33, 10], heads=2, seed=14, pad=30,
                               initial=torch.tensor([True, False]))
    for i in (0, 1, 2, 3, 4):
        args[i] = args[i].clone()
        args[i][43:] = float("nan")
    st = args[5]
    keep = int(args[7][0])
    for line in range(len(st)):
        if line != keep:
            st[line] = float("nan")
    out, got, want, want_st = run(args, kw)
    ref.check(out.cpu()[:43], want[:43], BF16, "out")
    for line in (keep, int(args[7][1])):
        ref.check(got.cpu()[line], want_st[line], F32, "state")


def test_split_calls_equal_one_call():
    """A sequence in two calls with the state carried, against one call."""
    args, kw = ref.rule_inputs([150], heads=2, dtype=F32, seed=30, initial=torch.tensor([True]))
    out, st, _, _ = run(args, kw)
    g = [to_gpu(a) for a in args]
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    parts = []
    for a, b in ((0, 61), (61, 62), (62, 150)):
        sub = [x[a:b] for x in g[:5]] + [g[5], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                         g[7], g[8]]
        parts.append(kd.gated_delta_rule_fn(*sub, **gkw, null_block_id=None))
    joined = torch.cat(parts)
    assert (joined - out).norm() <= 2 * ref.ARITHMETIC * out.norm()
    assert (g[5] - st).norm() <= 2 * ref.ARITHMETIC * st.norm()


@pytest.mark.parametrize("rate", [0.3, 0.7, 1.3, 3.0])
@pytest.mark.parametrize("lengths", [[900], [400, 1100, 9]], ids=str)
def test_fading_states(lengths, rate):
    """Decays that take a state, and what a stretch of tokens makes of the state before it,
    below FP32's range in some chunks; then values return, small or very large."""
    for dim in (64, 128):
        args, kw = ref.rule_inputs(lengths, heads=3, dim=dim, dtype=F32, gate="log", seed=31,
                                   initial=torch.ones(len(lengths), dtype=torch.bool))
        g = args[3]
        g[:, 0] = -rate
        g[:, 1] = -rate * torch.linspace(0.5, 1.5, dim)
        args[2][20:350, 2] = 0.0
        g[20:350, 2] = -rate
        compare(args, kw, f"rate {rate}")
        args[2][350:] *= 1e20
        compare(args, kw, f"rate {rate}, then large values")


@pytest.mark.parametrize("lengths", [[700], [1024, 5, 333], [2100]], ids=str)
def test_long_sequences(lengths):
    """Sequences long enough to be worked on in parts that run side by side."""
    for dim, gate, gd in ((128, "bounded", None), (64, "log", F32)):
        args, kw = ref.rule_inputs(lengths, heads=2, dim=dim, seed=7, gate=gate, gate_dtype=gd,
                                   initial=torch.ones(len(lengths), dtype=torch.bool))
        compare(args, kw)


def test_sequences_without_tokens():
    """They leave what they start from, whichever kernels a call takes."""
    for lengths in ([0, 40, 0, 0], [0, 3, 0, 0], [0] * 40 + [90], [2] * 30 + [0, 0]):
        initial = torch.arange(len(lengths)) % 2 == 0
        for dim in (64, 128):
            args, kw = ref.rule_inputs(lengths, heads=2, dim=dim, seed=9, initial=initial)
            before = args[5].clone()
            compare(args, kw, str(lengths))
            _, st, _, _ = run(args, kw)
            for s, n in enumerate(lengths):
                line = int(args[7][s])
                if n == 0:
                    assert torch.equal(st[line].cpu(), before[line] * float(initial[s]))


def test_many_short_sequences():
    gen = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 6, (500,), generator=gen).tolist()
    for dim in (64, 128):
        args, kw = ref.rule_inputs(lengths, heads=1, dim=dim, seed=2)
        compare(args, kw)


def mixed_lengths(short, most, long, seed):
    """`short` lengths of 0 to `most` tokens with the long ones spread among them."""
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, most + 1, (short,), generator=gen).tolist()
    for n in long:
        lengths.insert(int(torch.randint(0, len(lengths) + 1, (1,), generator=gen)), n)
    return lengths


@pytest.mark.parametrize("short,most,long,heads", [
    (70, 8, [500], 1),  # mostly short, few
    (150, 6, [300, 17, 16], 2),  # short on average
    (260, 30, [200, 33, 129], 8),  # not as short, many
    (4200, 2, [150], 1),  # more sequences than 64^2
], ids=str)
def test_short_and_long_together(short, most, long, heads):
    """Token-by-token and chunked sequences in one call, and the numbering of their pieces."""
    for at_end in (False, True):
        lengths = mixed_lengths(short, most, long, short)
        if at_end:
            lengths = sorted(lengths)
        args, kw = ref.rule_inputs(lengths, heads=heads, dim=64, seed=short, pad=2)
        compare(args, kw, f"sorted {at_end}")


@pytest.mark.parametrize("dtype,gate", [(BF16, "bounded"), (F16, "log"), (F32, "softplus")], ids=str)
def test_many_chunks(dtype, gate):
    """More chunks than get the larger workgroups."""
    lengths = [97, 33, 64, 129] * 8
    args, kw = ref.rule_inputs(lengths, heads=8, qk_heads=4, dim=128, dtype=dtype, gate=gate,
                               gate_dtype=F32 if gate == "log" else None, seed=12)
    compare(args, kw)


@pytest.mark.parametrize("dim", [64, 128])
def test_a_very_long_sequence(dim):
    """Nine thousand tokens through segment after segment."""
    args, kw = ref.rule_inputs([9001], heads=1, dim=dim, dtype=F32, gate="log", seed=41,
                               initial=torch.tensor([True]))
    compare(args, kw)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_segments(dim):
    """More segments than CUs."""
    args, kw = ref.rule_inputs([4096], heads=16, qk_heads=8, dim=dim, seed=43,
                               initial=torch.tensor([True]))
    compare(args, kw)


def test_far_rows():
    """Rows whose offset passes 2^31 elements: the widest token stride there is."""
    args, kw = ref.rule_inputs([290, 9], heads=1, dim=128, seed=42)
    stride, tokens = (1 << 23) - 8, 299
    big = torch.empty((tokens - 1) * stride + 4 * 128, dtype=BF16, device="cuda")
    g = [to_gpu(a) for a in args]
    for i in range(4):
        g[i] = big.as_strided((tokens, 1, 128), (stride, 128, 1), 128 * i)
        g[i].copy_(args[i])
    out = kd.gated_delta_rule_fn(*g, **{k: to_gpu(v) for k, v in kw.items()}, null_block_id=None)
    want, want_st = ref.delta_rule(*args, **kw)
    ref.check(out, want, BF16, "out")
    ref.check(g[5], want_st, F32, "states")
    one = [a[250:251] for a in g[:5]]
    before = g[5].clone()
    stepped = kd.gated_delta_rule_update(*one, g[5], g[7][:1], **{k: to_gpu(v) for k, v in kw.items()},
                                         null_block_id=None)
    args[5] = before.cpu()
    loc = torch.tensor([0, 1], dtype=torch.int32)
    want, want_st = ref.delta_rule(*[a[250:251] for a in args[:5]], args[5], loc, args[7][:1],
                                   torch.tensor([True]), **kw)
    ref.check(stepped, want, BF16, "step out")
    ref.check(g[5], want_st, F32, "step states")


def test_far_lines():
    """Lines whose offset passes 2^31 elements."""
    args, kw = ref.rule_inputs([40, 3], heads=1, dim=128, seed=17, lines=4,
                               initial=torch.tensor([True, True]))
    stride = 3 << 28
    big = torch.empty(3 * stride + 128 * 128, dtype=F32, device="cuda")
    st = big.as_strided((4, 1, 128, 128), (stride, 128 * 128, 128, 1))
    st.copy_(args[5])
    args[7] = torch.tensor([3, 1], dtype=torch.int32)
    g = [to_gpu(a) for a in args]
    g[5] = st
    out = kd.gated_delta_rule_fn(*g, **{k: to_gpu(v) for k, v in kw.items()}, null_block_id=None)
    want, want_st = ref.delta_rule(*args, **kw)
    ref.check(out, want, BF16, "out")
    ref.check(st.cpu(), want_st, F32, "states")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("batch", [1, 3, 70])
def test_update(batch, dtype, dim):
    args, kw = ref.rule_inputs([1] * batch, heads=3, dim=dim, dtype=dtype, seed=batch, strided=True,
                               initial=torch.ones(batch, dtype=torch.bool))
    if batch > 1:
        args[7][1] = 0
        args[7] = torch.where(torch.arange(batch) == 1, 0, torch.arange(batch) + 1).to(torch.int32)
    want, want_st = ref.delta_rule(*args, **kw, null_block_id=0)
    g = [to_gpu(a) for a in args]
    out = kd.gated_delta_rule_update(*g[:6], g[7], **{k: to_gpu(v) for k, v in kw.items()},
                                     null_block_id=0)
    ref.check(out, want, dtype, "out")
    ref.check(g[5], want_st, F32, "states")


def test_update_gates_and_strided_lines():
    for gate, per_head in (("log", True), ("softplus", False)):
        args, kw = ref.rule_inputs([1] * 9, heads=4, qk_heads=2, dim=128, gate=gate,
                                   per_head=per_head, gate_dtype=F32, beta_dtype=F32, seed=3,
                                   initial=torch.ones(9, dtype=torch.bool))
        want, want_st = ref.delta_rule(*args, **kw)
        g = [to_gpu(a) for a in args]
        lines = torch.stack([g[7], g[7] * 0 - 5], 1)[:, 0]  # stride 2
        out = kd.gated_delta_rule_update(*g[:6], lines, **{k: to_gpu(v) for k, v in kw.items()},
                                         null_block_id=None)
        ref.check(out, want, BF16, "out")
        ref.check(g[5], want_st, F32, "states")


def test_prefill_then_updates_continue_the_sequence():
    args, kw = ref.rule_inputs([64], heads=2, dtype=F32, seed=19, initial=torch.tensor([False]))
    want, want_st = ref.delta_rule(*args, **kw)
    g = [to_gpu(a) for a in args]
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    loc = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    out = [kd.gated_delta_rule_fn(*[x[:60] for x in g[:5]], g[5], loc, g[7], g[8], **gkw,
                                  null_block_id=None)]
    for t in range(60, 64):
        out.append(kd.gated_delta_rule_update(*[x[t:t + 1] for x in g[:5]], g[5], g[7], **gkw,
                                              null_block_id=None))
    ref.check(torch.cat(out), want, F32, "out")
    ref.check(g[5], want_st, F32, "states")


@pytest.mark.parametrize("lengths", [[130, 2, 50], [900]], ids=str)
def test_graph_replays(lengths):
    """Captured once, replayed with new values, lengths and lines of the same shapes; eager
    work between the replays."""
    args, kw = ref.rule_inputs(lengths, heads=2, seed=40)
    g = [to_gpu(a) for a in args]
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kd.gated_delta_rule_fn(*g, **gkw, null_block_id=None)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kd.gated_delta_rule_fn(*g, **gkw, null_block_id=None)
        step = kd.gated_delta_rule_update(*[x[:len(lengths)] for x in g[:5]], g[5], g[7], **gkw,
                                          null_block_id=None)
    total = sum(lengths)
    for seed in (41, 42, 43):
        other = list(lengths)
        if len(other) > 1:
            other[0], other[-1] = other[0] - 20, other[-1] + 20
        new, nkw = ref.rule_inputs(other, heads=2, seed=seed)
        for dst, src in zip(g, new):
            dst.copy_(src)
        for name in ("a_log", "dt_bias"):
            gkw[name].copy_(nkw[name])
        assert sum(other) == total
        eager = [x.clone() for x in g]
        graph.replay()
        torch.cuda.synchronize()
        want = kd.gated_delta_rule_fn(*eager, **gkw, null_block_id=None)
        want_step = kd.gated_delta_rule_update(*[x[:len(lengths)] for x in eager[:5]], eager[5],
                                               eager[7], **gkw, null_block_id=None)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(g[5], eager[5]) and torch.equal(step, want_step)


def test_side_stream_and_repeatable():
    args, kw = ref.rule_inputs([300, 40], heads=2, seed=50)
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    results = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        g = [to_gpu(a) for a in args]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            out = kd.gated_delta_rule_fn(*g, **gkw, null_block_id=None)
        stream.synchronize()
        results.append((out, g[5]))
    for out, st in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(st, results[0][1])


def test_empty_calls():
    args, kw = ref.rule_inputs([5], heads=2, seed=1)
    g = [to_gpu(a) for a in args]
    gkw = {k: to_gpu(v) for k, v in kw.items()}
    none = kd.gated_delta_rule_fn(*[x[:0] for x in g[:5]], g[5], g[6], g[7], g[8], **gkw)
    assert none.shape == (0, 2, 128)
    before = g[5].clone()
    kd.gated_delta_rule_fn(*g[:6], g[6][:1], g[7], g[8], **gkw)
    assert torch.equal(before, g[5])
    assert kd.gated_delta_rule_update(*[x[:0] for x in g[:5]], g[5], g[7], **gkw).shape == (0, 2, 128)
    assert kd.gated_delta_rule_supported(*g[:6])
    assert not kd.gated_delta_rule_supported(*g[:5], g[5].half())
