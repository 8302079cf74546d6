"""The precision of the weights of a shared prefix: 16 bits or more each, as in the attention of every sequence by
itself, however many rows share it; in longer chunks, as there, those of keys that hold much of a row's weight."""
import pytest
import torch

import adapter_linear_gb300 as al
import _kv_even_weights as E
import _kv_reference as R
import _kv_weights as W

pytestmark = pytest.mark.gpu

# Hq, H, D, page, prefix, sequences, new tokens of each (all its own)
CASES = [
    (8, 2, 128, 16, 1200, 4, 1),       # the short-chunk kernel
    (32, 8, 128, 16, 1104, 40, 1),     # the tcgen05 kernel, one tile
    (8, 1, 64, 32, 3000, 100, 2),      # several blocks of rows, items in pieces
    (4, 4, 128, 64, 1300, 70, 3),
    (16, 2, 64, 16, 2000, 3, 40),      # long chunks of their own: one part will do
    (4, 2, 128, 32, 1500, 5, [30, 1]), # beside short ones
]


@pytest.mark.parametrize("fmt", [al.LORA_KV_INT8, al.LORA_KV_BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights_of_a_prefix_keep_their_bits(case, fmt):
    Hq, H, D, page, pre, members, n = CASES[case]
    pre, new = pre // page * page, [n] * members if isinstance(n, int) else (n * members)[:members]
    p = R.Paged(al, fmt, [pre + x for x in new], new, H, D, page, seed=410 + case)
    p.table[1:, :pre // page] = p.table[0, :pre // page]
    K, V, Q = E.rows_on_eight_keys(p.T, pre, p.T, Hq, H, D, 400 + case, "cuda")

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    p.cache.write(K[:pre], V[:pre], al.KvBatch(p.table[:1].contiguous(), ints(0, pre), ints(pre), pre, pre))
    p.cache.write(K[pre:], V[pre:], p.batch)
    if fmt == al.LORA_KV_INT8:
        K, V = (q * s[..., None] for q, s in map(R.quantise, (K, V)))
    groups = al.KvGroups(ints(0, members), ints(pre), p.T)
    got, _ = p.cache.attention_shared(Q, p.batch, groups, scale=1.0)
    assert p.cache.check_errors() == al.LORA_OK
    long = min(new) * Hq // H > 24
    for b, n in enumerate(new):
        rows = slice(p.start[b], p.start[b] + n)
        own = slice(pre + p.start[b], pre + p.start[b] + n)
        k, v = (torch.cat((x[:pre], x[own])) for x in (K, V))
        O, A, S, A_rest = W.exact(Q[rows], k, v, torch.arange(pre + 1, pre + n + 1, device="cuda"))
        # the own keys score 0, 11 and more below the others: of a row's weight they hold n 2^-15 at most, which one
        # bf16 part may miss by 2^-8 of that, times the largest value
        rest = A_rest if long else n * 2.0 ** -15 * v[pre:].double().abs().amax()
        over = (got[rows].double() - O).abs() / W.bound(O, A, S, rest, pre + n)
        assert (over <= 1).all(), f"{CASES[case]}: {float(over.max()):.3g} of the bound"
