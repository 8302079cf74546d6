"""The bound that test_gpu_kv_weights.py holds the kernels to, on the CPU: weights in two bf16 parts meet it,
weights in one do not."""
import pytest
import torch

import _kv_reference as R
import _kv_weights as W


def rounded(w, parts):
    """w (float64) as the sum of `parts` bf16 numbers."""
    top = R.bf16_of_f64(w).double()
    return top if parts == 1 else top + R.bf16_of_f64(w - top).double()


@pytest.mark.parametrize("gap", [1, 32, 64, 300])
def test_the_bound_tells_one_part_from_two(gap):
    n, Hq, H, D, ctx = 12, 4, 2, 64, 640
    K, V, Q = W.rows_on_two_keys(n, Hq, H, D, ctx, gap, 5, "cpu")
    seen = torch.arange(ctx + 1, ctx + n + 1)
    O, A, S, A_rest = W.exact(Q, K, V, seen)
    limit = W.bound(O, A, S, A_rest, ctx + n)
    for parts in (1, 2):
        got = torch.zeros_like(O)
        for h in range(Hq):
            k, v = K[:, h // 2].double(), V[:, h // 2].double()
            z = Q[:, h].double() @ k.T
            z = z.masked_fill(torch.arange(ctx + n)[None, :] >= seen[:, None], float("-inf"))
            first = z.argmax(1, keepdim=True)                  # any number near the largest score
            w = torch.exp(z - torch.gather(z, 1, first) + 0.01)
            got[:, h] = rounded(w, parts) @ v / w.sum(1, keepdim=True)
        over = (R.bf16_of_f64(got).double() - O).abs() > limit
        assert over.any() == (parts == 1)
        if parts == 1:
            assert over.any(-1).double().mean() > 0.5           # of the rows, not a few elements
