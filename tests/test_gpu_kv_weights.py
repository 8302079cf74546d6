"""The softmax weights' precision: every weight of the short-chunk kernel, and those of keys that hold more
than a third of their row's weight in the tcgen05 kernel, have 16 bits or more on their way into the
product with V."""
import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R
import _kv_weights as W

pytestmark = pytest.mark.gpu

# Hq, H, D, page, new tokens, cached tokens, distance of the two keys
CASES = [
    (8, 2, 128, 16, 1, 600, 64),
    (8, 1, 64, 32, 1, 300, 1),
    (8, 2, 128, 64, 3, 900, 33),
    (8, 2, 64, 16, 5, 5000, 2000),
    (8, 2, 128, 32, 40, 300, 32),
    (4, 2, 64, 16, 70, 500, 1),
    (8, 1, 128, 16, 64, 700, 300),
    (4, 4, 128, 64, 150, 2000, 97),
    (16, 2, 64, 128, 33, 1200, 64),
]


@pytest.mark.parametrize("fmt", [al.LORA_KV_INT8, al.LORA_KV_BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights_that_matter_keep_their_bits(case, fmt):
    Hq, H, D, page, n, ctx, gap = CASES[case]
    K, V, Q = W.rows_on_two_keys(n, Hq, H, D, ctx, gap, 300 + case, "cuda")
    p = R.Paged(al, fmt, [ctx + n], [n], H, D, page, seed=310 + case)
    every = al.KvBatch(p.table, torch.tensor([0, ctx + n], dtype=torch.int32, device="cuda"), p.batch.kv_len,
                       ctx + n, ctx + n)
    p.cache.write(K, V, every)
    if fmt == al.LORA_KV_INT8:
        K, V = (q * s[..., None] for q, s in map(R.quantise, (K, V)))
    O, A, S, A_rest = W.exact(Q, K, V, torch.arange(ctx + 1, ctx + n + 1, device="cuda"))
    got, _ = p.cache.attention(Q, p.batch, scale=1.0)
    assert p.cache.check_errors() == al.LORA_OK
    over = (got.double() - O).abs() / W.bound(O, A, S, A_rest, ctx + n)
    assert (over <= 1).all(), f"{CASES[case]}: {float(over.max()):.3g} of the bound"
