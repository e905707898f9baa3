"""The operators of latent attention together: the example layer's chunks and decode steps."""

import importlib.util
import pathlib

import pytest
import torch

import latent_reference as ref

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "latent_layer", pathlib.Path(__file__).resolve().parent.parent / "examples" / "latent_layer.py")
latent_layer = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(latent_layer)


def tolerance(dtype, e4m3=False):
    """Of one way through the layer, relative to the output's norm. Roundings are of half a step u
    relative to each value and independent of one another. Queries pass three before a score
    (norm, projection, rotation or absorption) and keys three (projection, cache, up-projection):
    of channels of size one each moves a score by scale * sqrt(channels) u = u, and a weight by
    that much of itself. Values pass three as well, then come the weights', the result's and the
    output projections'. 12 in all, added up without their signs."""
    u = torch.finfo(dtype).eps / 2
    # A value one rounding away lies on another side of a boundary of 4 bits once in 2^-4 / u
    # times, and is then off by 2^-3: in keys and in values.
    flips = 2 * 2.0 ** -3 * (16 * u) ** 0.5 if e4m3 else 0.0
    return 12 * u + flips


def relative(got, want):
    return ((got.double().cpu() - want.double().cpu()).norm() / want.double().norm().cpu()).item()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("prompts,tokens,steps,kw", [
    (1, 9, 3, dict(page_size=1)), (3, 400, 5, {}), (2, 900, 2, dict(heads=8, page_size=16, factor=4.0)),
    (4, 300, 3, dict(heads=3, head_dim=64, rope_dim=32, latent=256, page_size=24))])
def test_chunks_and_decode_against_one_prefill(prompts, tokens, steps, kw, dtype, e4m3):
    stepped, whole, _ = latent_layer.compare(prompts, tokens, steps, dtype, e4m3=e4m3, **kw)
    assert bool(torch.isfinite(stepped).all())
    assert relative(stepped, whole) <= 2 * tolerance(dtype, e4m3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_against_its_definition(dtype):
    """Two chunks, expanded then absorbed, against FP64 on the CPU."""
    layer = latent_layer.LatentLayer(heads=2, head_dim=64, rope_dim=32, latent=128, hidden=256, pages=30, page_size=16,
                                     dtype=dtype)
    gen = torch.Generator().manual_seed(4)
    lengths, first = [70, 131], [66, 120]
    x = [torch.randn(n, 256, generator=gen).to(dtype) for n in lengths]
    residual = [torch.randn(n, 256, generator=gen).to(dtype) for n in lengths]
    table = torch.randperm(30, generator=gen)[:18].view(2, 9).to(torch.int32).cuda()

    def run(begin, end, form):
        seqs = torch.cat([torch.full((b - a,), s) for s, (a, b) in enumerate(zip(begin, end))]).cuda()
        positions = torch.cat([torch.arange(a, b) for a, b in zip(begin, end)]).cuda()
        rows = torch.cat([t[a:b] for t, a, b in zip(x, begin, end)]).cuda()
        res = torch.cat([t[a:b] for t, a, b in zip(residual, begin, end)]).cuda()
        slots, loc = layer.slots(table, seqs, positions), ref.starts([b - a for a, b in zip(begin, end)]).cuda()
        if form == "expanded":
            out = layer.prefill(rows, res, positions, slots, table, loc, ref.starts(end).cuda(), sum(end))
        else:
            out = layer.extend(rows, res, positions, slots, table, torch.tensor(end, dtype=torch.int32).cuda(), loc)
        return out.split([b - a for a, b in zip(begin, end)])

    parts = run([0, 0], first, "expanded"), run(first, lengths, "absorbed")

    def f64(t):
        return t.double().cpu()

    for s in range(2):
        h = f64(x[s]) + f64(residual[s])
        rows = ref.normed(h, f64(layer.norm_weight), layer.EPS) @ f64(layer.in_proj)
        pos = torch.arange(lengths[s])
        q = rows[:, :2 * 96].view(-1, 2, 96)
        q = torch.cat((q[..., :64], ref.turned(q[..., 64:], pos, layer.inv_freq.cpu(), False)), -1)
        latent = ref.normed(rows[:, 192:320], f64(layer.latent_weight), layer.EPS)
        rope = ref.turned(rows[:, 320:].unsqueeze(1), pos, layer.inv_freq.cpu(), False)[:, 0]
        up = (latent @ f64(layer.up_proj)).view(-1, 2, 128)
        o = ref.expanded(q, up[..., :64], rope, up[..., 64:], [0, lengths[s]], [0, lengths[s]], 96 ** -0.5)
        want = o.flatten(1) @ f64(layer.out_proj)
        for got, rows_of in ((parts[0][s], slice(0, first[s])), (parts[1][s], slice(first[s], None))):
            assert relative(got, want[rows_of]) <= tolerance(dtype), (s, rows_of)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_in_a_graph(e4m3):
    """A captured decode step over growing sequences, replayed with eager work between, against
    eager steps on another cache."""
    def make():
        return latent_layer.LatentLayer(heads=3, head_dim=64, rope_dim=32, latent=256, hidden=192, pages=12, page_size=4,
                                        e4m3=e4m3)

    eager, captured = make(), make()
    table = torch.arange(12, dtype=torch.int32).view(3, 4).cuda()
    seqs = torch.arange(3).cuda()
    x = torch.zeros(3, 192, dtype=torch.bfloat16, device="cuda")
    residual = torch.zeros_like(x)
    positions = torch.zeros(3, dtype=torch.int64, device="cuda")
    slots, lengths = captured.slots(table, seqs, positions), torch.ones(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.decode(x, residual, positions, slots, table, lengths)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.decode(x, residual, positions, slots, table, lengths)
    gen = torch.Generator().manual_seed(1)
    for i in range(7):
        tok, at = torch.randn(3, 192, generator=gen).bfloat16().cuda(), torch.tensor([i, i + 3, 2 * i]).cuda()
        x.copy_(tok)
        residual.zero_()
        positions.copy_(at)
        slots.copy_(captured.slots(table, seqs, at))
        lengths.copy_(at + 1)
        graph.replay()
        want = eager.decode(tok, torch.zeros_like(tok), at, eager.slots(table, seqs, at), table, (at + 1).to(torch.int32))
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_example_runs(capsys):
    latent_layer.main(["--prompts", "2", "--tokens", "130", "--steps", "2", "--cache", "e4m3"])
    assert "relative" in capsys.readouterr().out
