"""The example latent layer over a stretched context: the factor that rotary_frequencies gives
belongs to a whole score, of whose channels only a part is turned."""

import math

import pytest
import torch

import latent_reference as ref
from test_gpu_latent_example import latent_layer, relative, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_stretched_layer_against_its_definition(form):
    """One chunk, against FP64 on the CPU."""
    n, dtype = 90, torch.float16
    layer = latent_layer.LatentLayer(heads=2, head_dim=64, rope_dim=32, latent=128, hidden=256, pages=12, page_size=16,
                                     dtype=dtype, factor=8.0)
    gen = torch.Generator().manual_seed(4)
    x, residual = (torch.randn(n, 256, generator=gen).to(dtype) * 2 for _ in range(2))
    pos, table = torch.arange(n).cuda(), torch.arange(12, dtype=torch.int32)[None].cuda()
    slots, loc = layer.slots(table, torch.zeros_like(pos), pos), ref.starts([n]).cuda()
    if form == "expanded":
        got = layer.prefill(x.cuda(), residual.cuda(), pos, slots, table, loc, loc, n)
    else:
        got = layer.extend(x.cuda(), residual.cuda(), pos, slots, table, torch.tensor([n], dtype=torch.int32).cuda(), loc)

    def f64(t):
        return t.double().cpu()

    rows = ref.normed(f64(x) + f64(residual), f64(layer.norm_weight), layer.EPS) @ f64(layer.in_proj)
    f = layer.inv_freq.cpu()
    q = rows[:, :192].view(-1, 2, 96)
    q = torch.cat((q[..., :64], ref.turned(q[..., 64:], pos.cpu(), f, False)), -1)
    latent = ref.normed(rows[:, 192:320], f64(layer.latent_weight), layer.EPS)
    rope = ref.turned(rows[:, 320:].unsqueeze(1), pos.cpu(), f, False)[:, 0]
    up = (latent @ f64(layer.up_proj)).view(-1, 2, 128)
    temper = 0.1 * math.log(8.0) + 1  # of queries and of keys, all channels
    o = ref.expanded(q, up[..., :64], rope, up[..., 64:], [0, n], [0, n], 96 ** -0.5 * temper ** 2)
    # (Scores are as many times larger as their roundings.)
    assert relative(got, o.flatten(1) @ f64(layer.out_proj)) <= tolerance(dtype) * temper ** 2
