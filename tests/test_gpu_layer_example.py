"""The operators together: the example layer's prefill and decode."""

import importlib.util
import pathlib

import pytest
import torch

import rule_reference as ref

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "kda_layer", pathlib.Path(__file__).resolve().parent.parent / "examples" / "kda_layer.py")
kda_layer = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(kda_layer)

# Of an FP32 layer: four of the library's operators at 2^-17, and two products of up to 512
# terms whose FP32 sums may be off by 512 roundings of 2^-24 each: 2^-15 + 2 * 2^-15.
LAYER = 4 * ref.ARITHMETIC + 2 * 512 * 2.0 ** -24


def relative(got, want):
    return ((got.double().cpu() - want.double().cpu()).norm() / want.double().norm().cpu()).item()


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("prompts,tokens,steps", [(1, 5, 3), (3, 400, 5), (2, 900, 2)])
def test_decode_continues_prefill(prompts, tokens, steps, head_dim):
    stepped, whole, layer = kda_layer.compare(prompts, tokens, steps, torch.float32, 4, head_dim)
    assert relative(stepped, whole) <= 2 * LAYER
    assert relative(layer.states[:prompts], layer.states[prompts:]) <= 2 * LAYER
    # The same inputs went into both conv states; only the projections' row counts differ.
    assert relative(layer.conv_states[:prompts], layer.conv_states[prompts:]) <= LAYER


def test_layer_against_its_definition():
    """Prefill against FP64 on the CPU."""
    layer = kda_layer.KdaLayer(heads=2, head_dim=64, hidden=256, lines=2, dtype=torch.float32)
    lengths = [70, 131]
    T = sum(lengths)
    gen = torch.Generator().manual_seed(4)
    x, residual = torch.randn(T, 256, generator=gen), torch.randn(T, 256, generator=gen)
    qsl = torch.tensor([0, 70, 201], dtype=torch.int32)
    lines = torch.tensor([1, 0], dtype=torch.int32)
    new = torch.zeros(2, dtype=torch.bool)
    res = residual.cuda()
    got = layer.prefill(x.cuda(), res, qsl.cuda(), lines.cuda(), new.cuda())

    def f64(t):
        return t.double().cpu()

    h = f64(x) + f64(residual)
    assert relative(res, h) <= 2.0 ** -24
    y = h / (h.square().mean(-1, keepdim=True) + layer.EPS).sqrt() * f64(layer.norm_weight)
    rows = y @ f64(layer.in_proj)
    qkv, gate, out_gate, beta = layer._columns(rows)
    conv = torch.zeros_like(qkv)
    w = f64(layer.conv_weight)
    for a, b in zip(qsl[:-1].tolist(), qsl[1:].tolist()):
        padded = torch.cat([torch.zeros(3, qkv.shape[1], dtype=torch.float64), qkv[a:b]])
        conv[a:b] = sum(padded[i:i + b - a] * w[:, i] for i in range(4))
    conv = conv * torch.sigmoid(conv)
    q, k, v = (t.unflatten(1, (2, 64)) for t in conv.split(128, 1))
    o, states = ref.delta_rule(q, k, v, gate, beta, torch.zeros(2, 2, 64, 64, dtype=torch.float64),
                               qsl, lines, new, a_log=f64(layer.a_log), dt_bias=f64(layer.dt_bias),
                               lower_bound=-5.0, beta_logits=True, null_block_id=None)
    o = o / (o.square().mean(-1, keepdim=True) + layer.EPS).sqrt() * f64(layer.head_weight)
    o = o * torch.sigmoid(out_gate)
    want = o.reshape(T, 128) @ f64(layer.out_proj)
    assert relative(got, want) <= LAYER
    assert relative(layer.states, states) <= LAYER


def test_decode_in_a_graph():
    """A captured decode step, replayed with eager work between, against eager steps."""
    def make():
        torch.manual_seed(0)
        layer = kda_layer.KdaLayer(heads=3, head_dim=64, hidden=192, lines=5)
        layer.states.normal_(std=0.3)
        layer.conv_states.normal_(std=0.3)
        return layer

    eager, captured = make(), make()
    lines = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    x = torch.zeros(3, 192, dtype=torch.bfloat16, device="cuda")
    residual = torch.zeros_like(x)
    steps = [torch.randn(3, 192, device="cuda").bfloat16() for _ in range(5)]
    keep = captured.states.clone(), captured.conv_states.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.decode(x, residual, lines)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.decode(x, residual, lines)
    captured.states.copy_(keep[0])
    captured.conv_states.copy_(keep[1])
    for tok in steps:
        x.copy_(tok)
        residual.zero_()
        graph.replay()
        want = eager.decode(tok, torch.zeros_like(tok), lines)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(captured.states, eager.states)
