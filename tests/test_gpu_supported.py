"""Queries of support take no memory on the GPU and run nothing there."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu


def test_supported_allocates_nothing():
    cache = ref.on_gpu(*ref.cache(4, 16, 512, 64, torch.bfloat16))
    q = torch.zeros(300, 16, 512 + 64, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros(2, 500, 16, 128, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros(500, 64, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    with torch.cuda.stream(stream):
        assert kd.latent_attention_supported(q[..., :512], q[..., 512:], *cache)
        assert not kd.latent_attention_supported(q[..., :504], q[..., 512:], *cache)
        assert kd.expanded_attention_supported(q[..., :192], k, kr, v)
        assert not kd.expanded_attention_supported(q[..., :192], k, None, v)
        assert kd.latent_attention_supported(q[:0, :, :512], q[:0, :, 512:], *cache)
        assert kd.expanded_attention_supported(q[:0, :, :192], k[:0], kr[:0], v[:0])
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_supported_in_a_capture():
    """Where work may be recorded, too."""
    cache = ref.on_gpu(*ref.cache(4, 16, 512, 64, torch.bfloat16))
    q = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        assert kd.latent_attention_supported(q[..., :512], q[..., 512:], *cache)
        out = kd.latent_attention_update(q[..., :512], q[..., 512:], *cache, table, lens, scale=0.1)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kd.latent_attention_update(q[..., :512], q[..., 512:], *cache, table, lens, scale=0.1))
