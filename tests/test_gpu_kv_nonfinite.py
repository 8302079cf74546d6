"""Infinities and NaN among an unquantised cache's tokens: they belong to the rows that see them."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

# Hq, H, D, page, lens, new, window, tokens with a bad value (sequence, position)
CASES = [
    (8, 2, 128, 16, [200, 40], [3, 1], 0, [(0, 199), (0, 198)]),             # inside short chunks
    (8, 2, 128, 16, [500], [1], 100, [(0, 399), (0, 390)]),                  # just outside a window
    (8, 4, 64, 16, [300, 90], [4, 2], 50, [(0, 248), (1, 38), (1, 89)]),     # at a window's edge
    (24, 1, 64, 32, [130], [1], 64, [(0, 65), (0, 3)]),
    (8, 2, 128, 64, [400], [300], 0, [(0, 250), (0, 399)]),                  # inside long chunks
    (4, 1, 64, 16, [700, 60], [260, 60], 90, [(0, 500), (0, 420), (1, 59)]),
    (8, 8, 128, 32, [1500], [128], 700, [(0, 690), (0, 1450)]),
]


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_bad_value_of_v_stays_with_the_rows_that_see_it(case, value):
    Hq, H, D, page, lens, new, window, bad = CASES[case]
    p = R.Paged(al, al.LORA_KV_BF16, lens, new, H, D, page, seed=70 + case)
    Q = torch.randn(p.T, Hq, D, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(D), window)      # with the values that were there before
    dim = 37
    for b, pos in bad:
        pg, r = p.where(b, torch.tensor([pos], device="cuda"))
        p.cache.v[pg, :, r, dim] = value
    O, lse = p.cache.attention(Q, p.batch, window=window)
    assert p.cache.check_errors() == al.LORA_OK
    sees = torch.zeros(p.T, dtype=torch.bool, device="cuda")
    for b, at in bad:
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        sees[p.start[b]:p.start[b + 1]] |= (at <= pos) & ((at > pos - window) if window else (pos >= 0))
    assert bool(sees.any()) or case in (1, 3)
    assert not torch.isfinite(O[sees][:, :, dim]).any()
    R.check_attention(O[~sees], lse[~sees], tuple(x[~sees] for x in ref), f"{CASES[case]}")
    others = [d for d in range(D) if d != dim]
    R.check_attention(O[..., others], lse, (ref[0][..., others], ref[1], ref[2][..., others], ref[3]), f"{CASES[case]}")


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_bad_key_stays_with_the_rows_that_see_it(case):
    Hq, H, D, page, lens, new, window, bad = CASES[case]
    p = R.Paged(al, al.LORA_KV_BF16, lens, new, H, D, page, seed=90 + case)
    Q = torch.randn(p.T, Hq, D, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(D), window)
    sees = torch.zeros(p.T, dtype=torch.bool, device="cuda")
    for b, at in bad:
        pg, r = p.where(b, torch.tensor([at], device="cuda"))
        p.cache.k[pg, :, r] = float("nan")
        p.cache.v[pg, :, r] = float("nan")
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        sees[p.start[b]:p.start[b + 1]] |= (at <= pos) & ((at > pos - window) if window else (pos >= 0))
    O, lse = p.cache.attention(Q, p.batch, window=window)
    assert p.cache.check_errors() == al.LORA_OK
    assert torch.isnan(O[sees].float()).all() and torch.isnan(lse[sees]).all()
    R.check_attention(O[~sees], lse[~sees], tuple(x[~sees] for x in ref), f"{CASES[case]}")
