"""Scores that rise, fall or jump inside a tile of keys: the running maximum moves at every place it
can, or never again."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

L = 700


def shapes():
    j = torch.arange(L, device="cuda").double()
    return {
        "rise": 0.6 * j,                                  # 32 keys raise the maximum by 2^28
        "slow": 0.05 * j,
        "fall": -0.6 * j,
        "jump": 40.0 * (j >= 70) + 40.0 * (j >= 300),     # in the second half of a tile
        "steps": 15.0 * torch.floor(j / 32),              # just under and
        "higher": 19.0 * torch.floor(j / 32),             # over what moves the maximum
        "alternate": 60.0 * (j.long() // 32 % 2),
        "huge": 3.0e4 * (j == 333),
    }


@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("shape", sorted(["rise", "slow", "fall", "jump", "steps", "higher", "alternate", "huge"]))
@pytest.mark.parametrize("fmt", [al.LORA_KV_BF16, al.LORA_KV_INT8])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_along_the_keys(D, fmt, shape, new):
    H, Hq = 2, 8
    p = R.Paged(al, fmt, [L], [new], H, D, 16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    # one dimension carries the wanted score, the others add noise
    x = torch.randn(L, H, D, generator=g, device="cuda") * 0.1
    x[..., 3] = (shapes()[shape] / 8.0).float()[:, None]
    x = x.to(torch.bfloat16)
    pages, rows = p.where(0, torch.arange(L, device="cuda"))
    if fmt == al.LORA_KV_INT8:
        q, s = R.quantise(x)
        p.cache.k[pages, :, rows] = q.to(torch.int8)
        p.cache.k_scales[pages, :, rows] = s.to(torch.bfloat16)
        p.values[0][0] = q * s[..., None]
    else:
        p.cache.k[pages, :, rows] = x
        p.values[0][0] = x.double()
    Q = torch.randn(new, Hq, D, generator=g, device="cuda")
    Q[..., 3] = 8.0
    Q = Q.to(torch.bfloat16)
    O, lse = p.cache.attention(Q, p.batch, scale=1.0)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, 1.0), f"{shape} {new} {D}")
