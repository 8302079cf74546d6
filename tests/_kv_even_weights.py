"""Rows whose weight lies on eight keys, an eighth each or so, whose values nearly cancel: no key holds much of a row's
weight once four are counted, and the rounding of the others' weights shows in O."""
import torch

KEYS = 8


def keys_of(a):
    """The keys that answer to dimension a: four, and four 32 behind them, of 64 tokens."""
    i = torch.arange(KEYS)
    return 64 * a[:, None] + i % 4 + 32 * (i // 4)


def rows_on_eight_keys(rows, ctx, own, Hq, H, D, seed, device):
    """K, V [ctx + own][H][D] and Q [rows][Hq][D] (bf16): query (t, h) asks for a dimension, its eight keys answer, all
    others score 0. ctx >= 64."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    n = min(D, ctx // 64)
    K, V = torch.zeros(ctx + own, H, D), torch.randn(ctx + own, H, D, generator=g)
    a = torch.arange(n)
    at = keys_of(a)
    for i in range(KEYS):
        K[at[:, i], :, a] = torch.rand(n, H, generator=g) * 0.02 + 0.99
        V[at[:, i]] = V[at[:, 0]] * (-1) ** i
    Q = torch.zeros(rows, Hq, D)
    ask = torch.randint(0, n, (rows, Hq, 1), generator=g)
    Q.scatter_(2, ask, torch.rand(rows, Hq, 1, generator=g) * 4 + 12)
    return tuple(x.to(torch.bfloat16).to(device) for x in (K, V, Q))
