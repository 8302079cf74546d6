"""8-bit caches, chunks whose row blocks alternate between one and two 128-row tiles, and more work
than one block an SM: a CTA goes from blocks of one tile to blocks of two, over many key tiles. The
values' scales differ by powers of two from key tile to key tile, so that a scale of another tile's
keys shows."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

# sequences, new tokens in turn, cached tokens, Hq, H, D, page
CASES = [
    (24, (20, 64), 1500, 32, 8, 128, 16),      # 80 rows: one tile; 256: two
    (150, (20, 64), 1000, 4, 1, 128, 16),
    (160, (5, 40, 33), 700, 16, 2, 64, 32),    # 40, 320 and 264 rows: last blocks of 64 and 8
    (100, (70, 81), 900, 14, 2, 128, 64),      # 490 and 567 rows: last blocks of 234 and 55
    (200, (12, 32), 800, 8, 1, 64, 16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_blocks_of_one_and_two_tiles_in_turn(case):
    n, turn, ctx, Hq, H, D, page = CASES[case]
    new = [turn[b % len(turn)] for b in range(n)]
    lens = [ctx + 37 * (b % 11) + m for b, m in enumerate(new)]
    p = R.Paged(al, al.LORA_KV_INT8, lens, new, H, D, page, seed=130 + case)
    for b, L in enumerate(lens):
        pos = torch.arange(L, device="cuda")
        up = 2.0 ** ((pos // 128 * 5) % 9 - 4).double()
        pages, rows = p.where(b, pos)
        p.cache.v_scales[pages, :, rows] = (p.cache.v_scales[pages, :, rows].double() * up[:, None]).to(torch.bfloat16)
        p.values[b][1] = p.values[b][1] * up[:, None, None]
    g = torch.Generator(device="cuda").manual_seed(case)
    Q = torch.randn(p.T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    O, lse = p.cache.attention(Q, p.batch)
    assert p.cache.check_errors() == al.LORA_OK
    R.check_attention(O, lse, R.attention(Q, p, 1.0 / math.sqrt(D)), f"{CASES[case]}")
    for _ in range(50):
        O2, lse2 = p.cache.attention(Q, p.batch)
        assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(lse, lse2)
    assert p.cache.check_errors() == al.LORA_OK
