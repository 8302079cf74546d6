"""Infinities and NaN among an unquantised cache's values: a row that sees one has that infinity there, NaN
with a NaN or infinities of both signs, whatever the token's weight and wherever it lies; the other
dimensions and rows are what they were."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# Hq, H, D, page, lens, new, window, bad values (sequence, position, dimension, value)
CASES = [
    # single tokens: far from the end, at the end, both signs, a NaN
    (8, 2, 128, 16, [300, 70], [1, 1], 0, [(0, 17, 3, INF), (0, 299, 4, -INF), (0, 80, 5, INF), (0, 90, 5, -INF),
                                           (1, 0, 64, NAN), (1, 69, 127, INF)]),
    (24, 2, 64, 32, [900], [2], 0, [(0, 5, 63, -INF), (0, 898, 0, INF), (0, 899, 0, -INF), (0, 899, 1, INF)]),
    (8, 8, 64, 16, [5000, 3000], [3, 1], 700, [(0, 4500, 9, INF), (0, 4297, 10, INF), (0, 4298, 11, -INF),
                                              (0, 100, 12, INF), (1, 2300, 13, NAN), (1, 2299, 14, NAN)]),
    # split over many CTAs
    (4, 1, 128, 64, [40000], [1], 0, [(0, 1, 2, INF), (0, 20000, 3, -INF), (0, 39999, 2, INF), (0, 7, 3, INF)]),
    # long chunks: seen by all rows, inside the chunk, outside a window, both
    (8, 2, 128, 64, [700], [300], 0, [(0, 10, 1, INF), (0, 390, 2, -INF), (0, 550, 3, INF), (0, 20, 3, -INF),
                                      (0, 699, 4, NAN), (0, 200, 5, INF), (0, 650, 5, INF)]),
    (16, 2, 64, 32, [2000, 150], [200, 150], 400, [(0, 1500, 1, INF), (0, 1700, 2, -INF), (0, 100, 3, INF),
                                                   (0, 1401, 4, INF), (0, 1999, 5, NAN), (1, 0, 6, INF)]),
    (8, 1, 128, 16, [30000, 60], [40, 60], 0, [(0, 3, 100, -INF), (0, 29000, 101, INF), (0, 29980, 101, INF),
                                               (0, 15000, 102, INF), (0, 15001, 102, -INF), (1, 30, 7, INF)]),
]


@pytest.mark.parametrize("scale", [None, 5.0])      # 5: most weights are 0 in fp32
@pytest.mark.parametrize("case", range(len(CASES)))
def test_bad_values_reach_the_rows_that_see_them_as_they_are(case, scale):
    Hq, H, D, page, lens, new, window, bad = CASES[case]
    p = R.Paged(al, al.LORA_KV_BF16, lens, new, H, D, page, seed=270 + case)
    g = torch.Generator(device="cuda").manual_seed(case)
    Q = torch.randn(p.T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ref = R.attention(Q, p, scale, window)           # with the values that were there before
    want = torch.zeros(p.T, D, dtype=torch.float64, device="cuda")
    for b, at, dim, value in bad:
        pages, rows = p.where(b, torch.tensor([at], device="cuda"))
        p.cache.v[pages, :, rows, dim] = value
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        sees = (at <= pos) & ((at > pos - window) if window else (pos >= 0))
        want[p.start[b]:p.start[b + 1], dim] += torch.where(sees, value, 0.0)
    O, lse = p.cache.attention(Q, p.batch, scale=scale, window=window)
    assert p.cache.check_errors() == al.LORA_OK
    hit = (want != 0)[:, None, :].expand(O.shape)
    want = want.to(torch.bfloat16)[:, None, :].expand(O.shape)
    assert hit.any()
    assert torch.equal(torch.isnan(O[hit]), torch.isnan(want[hit]))
    sign = hit & ~torch.isnan(want)
    assert torch.equal(O[sign], want[sign])
    clean = torch.where(hit, ref[0], O.double())      # the rest against 64 bits
    R.check_attention(clean, lse, ref, f"{CASES[case][:7]}")
    O2, lse2 = p.cache.attention(Q, p.batch, scale=scale, window=window)
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [[1, 2], [60, 40]])
def test_rows_whose_query_is_not_a_number(new):
    """They are NaN throughout, and the others find an infinity of V all the same."""
    p = R.Paged(al, al.LORA_KV_BF16, [500, 900], new, 2, 128, 32, seed=290)
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(128))
    Q[1, 2, 5] = NAN
    pages, rows = p.where(1, torch.tensor([12], device="cuda"))
    p.cache.v[pages, :, rows, 77] = -INF
    O, lse = p.cache.attention(Q, p.batch)
    nan = torch.zeros(p.T, 8, dtype=torch.bool, device="cuda")
    nan[1, 2] = True
    assert torch.isnan(O[nan]).all() and torch.isnan(lse[nan]).all()
    keep = ~nan
    got = O.double()
    assert (got[p.start[1]:, :, 77][keep[p.start[1]:]] == -INF).all()
    got[p.start[1]:, :, 77] = ref[0][p.start[1]:, :, 77]
    R.check_attention(got[keep], lse[keep], tuple(x[keep] for x in ref), f"{new}")
