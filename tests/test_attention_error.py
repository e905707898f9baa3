"""The bound on a row's error (attention_error) on the CPU: rounded weights and results pass it,
a lost or doubled step of keys does not, at the longest lengths that the kernels are tested at."""

import pytest
import torch

import attention_error as ae
import latent_reference as ref

BF16, F16 = torch.bfloat16, torch.float16


def normal(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def rounded(scores, values, dtype):
    """Weights rounded to dtype before their sum's division, one rounding of the result."""
    w = torch.exp2((scores - scores.amax(-1, keepdim=True)) * 1.4426950408889634)
    return ((w.to(dtype).double() @ values) / w.sum(-1, keepdim=True)).to(dtype).double()


CASES = pytest.mark.parametrize("form,keys,step", [("absorbed", 20000, 32), ("absorbed", 9000, 32), ("expanded", 9000, 64),
                                                   ("expanded", 7000, 64)])


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@CASES
def test_bound(form, keys, step, dtype):
    """Scores and values as the GPU tests make them (see flat there)."""
    channels, rope = (256, 64) if form == "absorbed" else (128, 64)
    k, r = normal(keys, channels, dtype=dtype).double(), normal(keys, rope, seed=1, dtype=dtype).double()
    v = k if form == "absorbed" else normal(keys, channels, seed=2, dtype=dtype).double()
    q = normal(12, channels + rope, seed=3, dtype=dtype).double()
    for scale in (0.02, 192 ** -0.5):
        w = (q[:, :channels] @ k.T + q[:, channels:] @ r.T) * scale
        seen = torch.ones_like(w, dtype=torch.bool)
        out, spread = ae.rows(w, seen, v)
        assert ae.worst(rounded(w, v, dtype), out, spread, dtype) < 1
        if scale > 0.05:
            continue
        for first in range(0, keys - step, keys // 40):
            lost = w.clone()
            lost[:, first:first + step] = -1e30
            assert ae.worst(rounded(lost, v, dtype), out, spread, dtype) > 1, ("lost", first)
            twice = torch.cat([w, w[:, first:first + step]], -1)
            assert ae.worst(rounded(twice, torch.cat([v, v[first:first + step]]), dtype), out, spread, dtype) > 1, ("twice", first)


def test_rows_are_the_reference():
    """attention_error's rows are those of latent_reference."""
    table, pages = ref.tables([40, 9], 8)
    cache = ref.cache(pages, 8, 64, 16, BF16)
    q, r, loc = normal(5, 3, 64, dtype=BF16), normal(5, 3, 16, seed=1, dtype=BF16), ref.starts([3, 2])
    args = (q, r, cache, table, torch.tensor([40, 9]), loc, 0.1)
    assert torch.allclose(ae.absorbed(*args)[0], ref.attention(q, r, *cache, *args[3:]), atol=1e-12)
    kv, kr = normal(50, 3, 96, seed=2, dtype=BF16), normal(50, 16, seed=3, dtype=BF16)
    q, kv_loc = normal(5, 3, 80, seed=4, dtype=BF16), ref.starts([40, 10])
    for causal in (True, False):
        args = (q, kv[..., :64], kr, kv[..., 64:], loc, kv_loc, 0.1, causal)
        assert torch.allclose(ae.expanded(*args)[0], ref.expanded(*args), atol=1e-12)
