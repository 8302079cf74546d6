"""Rows whose weight lies on two keys with opposite values, so that O is small beside what it is summed
from and a weight's rounding shows; and the bound that holds if those two weights have 16 bits or more."""
import torch


def rows_on_two_keys(n, Hq, H, D, ctx, gap, seed, device):
    """K, V [ctx + n][H][D] and Q [n][Hq][D] (bf16): query (t, h) asks for dimension a; keys a and a + gap
    answer, all others score 0. a + gap < ctx: every row sees both."""
    g = torch.Generator(device="cpu").manual_seed(seed)

    def uniform(*shape, lo, hi):
        return torch.rand(*shape, generator=g) * (hi - lo) + lo

    keys = min(D, gap, ctx - gap)
    K = torch.zeros(ctx + n, H, D)
    a = torch.arange(keys)
    K[a, :, a] = 1.0
    K[a + gap, :, a] = uniform(keys, H, lo=0.98, hi=1.02)
    V = torch.randn(ctx + n, H, D, generator=g)
    V[a + gap] = -V[a]
    Q = torch.zeros(n, Hq, D)
    ask = torch.randint(0, keys, (n, Hq, 1), generator=g)
    Q.scatter_(2, ask, uniform(n, Hq, 1, lo=12.0, hi=16.0))
    return tuple(x.to(torch.bfloat16).to(device) for x in (K, V, Q))


def bound(O, A, S, A_rest, keys):
    """For scale 1. O, A, S as in _kv_reference.attention; A_rest: the part of A of the keys with at most a
    third of their row's weight.
    - the output's rounding, 2^-8 |O|;
    - a weight in two bf16 parts, 2^-8 2^-8 of it; in one, 2^-8 (the other keys');
    - a dot product of one term is exact; its factors (the scale's log2 e, a key's scale), the difference from m
      and exp2 lose less than 2^-22 (2 + S) of a weight, which moves O by at most twice that times A;
    - fp32 sums over the keys, 16 at a time, twice, each losing 2^-22 of at most A."""
    steps = 2 * (keys / 16 + 8)
    loss = 2.0 ** -16 + 2 * 2.0 ** -22 * (2 + S[..., None]) + steps * 2.0 ** -22
    return 2.0 ** -8 * O.abs() + A * loss + 2.0 ** -8 * A_rest + 2.0 ** -100


def exact(Q, K, V, visible):
    """(O, A, S, A_rest) in float64, K and V [keys][H][D] as the cache holds them, scale 1; visible: a
    number of keys per row of Q."""
    n, Hq, D = Q.shape
    G = Hq // K.shape[1]
    out = [torch.zeros(n, Hq, D, dtype=torch.float64, device=Q.device) for _ in range(3)]
    S = torch.zeros(n, Hq, dtype=torch.float64, device=Q.device)
    hidden = torch.arange(K.shape[0], device=Q.device)[None, :] >= visible[:, None]
    for h in range(Hq):
        k, v = K[:, h // G].double(), V[:, h // G].double()
        z = (Q[:, h].double() @ k.T).masked_fill(hidden, float("-inf"))
        p = torch.softmax(z, 1)
        rest = torch.where(p > 1 / 3, torch.zeros_like(p), p)
        for x, w in zip(out, (p @ v, p @ v.abs(), rest @ v.abs())):
            x[:, h] = w
        S[:, h] = z.masked_fill(hidden, 0).abs().amax(1)
    return out[0], out[1], S, out[2]
