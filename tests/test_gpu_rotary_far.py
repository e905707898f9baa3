"""Rotary positions past 2^29, where position times frequency is no longer exact in FP64."""

import pytest
import torch

import latent_reference as ref
import packed_varlen_causal_depthwise_amd as kd

pytestmark = pytest.mark.gpu

FAR = [1 << 29, (1 << 29) + 1, (1 << 31) - 1, (1 << 31) + 12345, (1 << 40) + 987654321, -(1 << 40) - 3, (1 << 47) + 1234567,
       (1 << 53) - 1, -(1 << 53) + 1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_far_positions(interleaved):
    """Against 300-bit arithmetic: as near as any other position."""
    from mpmath import cos, mp, mpf, sin

    mp.prec = 300
    f = ref.frequencies(64)
    x = torch.zeros(len(FAR), 1, 64)
    first = slice(0, None, 2) if interleaved else slice(0, 32)
    second = slice(1, None, 2) if interleaved else slice(32, None)
    x[..., first] = 1.0
    got = kd.rotary_embedding(x.cuda(), torch.tensor(FAR).cuda(), f.cuda(), interleaved=interleaved).cpu().double()
    for i, p in enumerate(FAR):
        for j, w in enumerate(f.tolist()):
            a = mpf(p) * mpf(w)
            # An angle off by 2^-26 of a turn is 1.6 * 2^-24; sine and cosine 2 units of 2^-24 each.
            assert abs(float(cos(a)) - got[i, 0, first][j]) < 8 * 2.0 ** -24, (p, j)
            assert abs(float(sin(a)) - got[i, 0, second][j]) < 8 * 2.0 ** -24, (p, j)


def test_cache_write_far_positions():
    """The cache's rotated parts turn alike."""
    pos, f = torch.tensor(FAR).cuda(), ref.frequencies(64).cuda()
    n = len(FAR)
    r = torch.randn(n, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    latents = torch.zeros(1, n, 64, dtype=torch.bfloat16, device="cuda")
    ropes = torch.zeros_like(latents)
    kd.latent_cache_write(r, r, latents, ropes, None, torch.arange(n).cuda(), positions=pos, inv_freq=f)
    assert torch.equal(ropes[0], kd.rotary_embedding(r[:, None], pos, f)[:, 0])
