"""The norms' kernels against their definition in FP64 (rule_reference)."""

import pytest
import torch

import packed_varlen_causal_depthwise_amd as kd
import rule_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def normal(*shape, seed=0, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 8), (1, 12, 128), (7, 3, 64), (37, 5, 192),
                                              (3, 2, 512), (130, 12, 128), (9, 1, 72), (5000, 9, 64)])
def test_gated(tokens, heads, dim, dtype):
    x, z = (normal(tokens, heads, dim, seed=s, dtype=dtype) for s in (1, 2))
    w = normal(dim, seed=3) + 1
    for act in ("sigmoid", "silu"):
        got = kd.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), activation=act, eps=1e-5)
        ref.check(got, ref.gated_norm(x, z, w, 1e-5, act), dtype, act)
    got = kd.gated_rms_norm(x.cuda(), None, None, eps=0.5)
    ref.check(got, ref.gated_norm(x, None, None, 0.5, ""), dtype, "plain")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_gated_strides_and_in_place(dtype):
    rows = normal(70, 900, seed=4, dtype=dtype).cuda()
    x = rows[:, 1:1 + 4 * 64].unflatten(1, (4, 64))
    z = rows[:, 301:301 + 4 * 128].unflatten(1, (4, 128))[..., :64]
    want = ref.gated_norm(x.cpu(), z.cpu(), None, 1e-5, "silu")
    ref.check(kd.gated_rms_norm(x, z, None, activation="silu"), want, dtype, "strided")
    y = x.contiguous()
    got = kd.gated_rms_norm(y, z, None, activation="silu", out=y)
    assert got is y
    ref.check(y, want, dtype, "in place")


def test_gated_extremes():
    x = normal(4, 2, 64, seed=5)
    z = torch.full_like(x, 200.0)
    z[1] = -200.0
    z[2] = 0.0
    x[3] = 0.0
    for act in ("sigmoid", "silu"):
        got = kd.gated_rms_norm(x.cuda(), z.cuda(), None, activation=act)
        ref.check(got, ref.gated_norm(x, z, None, 1e-5, act), F32, act)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("tokens,hidden", [(1, 1), (3, 7), (2, 8), (5, 513), (4, 1000), (37, 2048),
                                           (6, 4096), (3, 4097), (2, 8192), (2, 16384), (3, 12345),
                                           (2000, 576)])
def test_residual(tokens, hidden, dtype):
    x, r = (normal(tokens, hidden, seed=s, dtype=dtype) for s in (1, 2))
    w = normal(hidden, seed=3) + 1
    for residual, weight, scale in ((r, w, 0.25), (r, None, 1.0), (None, w, 2.0)):
        want, h = ref.residual_norm(x, residual, weight, 1e-5, scale)
        res = None if residual is None else residual.cuda()
        got = kd.residual_rms_norm(x.cuda(), res, None if weight is None else weight.cuda(),
                                   residual_scale=scale)
        ref.check(got, want, dtype, "out")
        if res is not None:
            ref.check(res, h, dtype, "residual")


def test_residual_strides():
    wide = normal(20, 700, seed=6, dtype=BF16).cuda()
    x, r = wide[:, 3:303], wide[:, 351:651]
    keep = wide.clone()
    want, h = ref.residual_norm(x.cpu(), r.cpu(), None, 1e-6, 0.5)
    got = kd.residual_rms_norm(x, r, None, eps=1e-6, residual_scale=0.5)
    ref.check(got, want, BF16, "out")
    ref.check(r, h, BF16, "residual")
    assert torch.equal(wide[:, :351], keep[:, :351]) and torch.equal(wide[:, 651:], keep[:, 651:])


def test_norms_in_a_graph():
    x, z, r = (normal(50, 256, seed=s, dtype=BF16).cuda() for s in (1, 2, 3))
    shape = (50, 2, 128)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = kd.gated_rms_norm(x.view(shape), z.view(shape), None)
        out = kd.residual_rms_norm(y.view(50, 256), r, None)
    for seed in (4, 5, 6):
        x.copy_(normal(50, 256, seed=seed, dtype=BF16))
        start = r.clone()
        graph.replay()
        torch.cuda.synchronize()
        e = kd.gated_rms_norm(x.view(shape), z.view(shape), None)
        want = kd.residual_rms_norm(e.view(50, 256), start, None)
        assert torch.equal(out, want) and torch.equal(r, start)


def test_empty():
    assert kd.gated_rms_norm(torch.empty(0, 2, 64, device="cuda"), None, None).shape == (0, 2, 64)
    assert kd.residual_rms_norm(torch.empty(0, 64, device="cuda"), None, None).shape == (0, 64)
