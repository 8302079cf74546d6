"""The bound that test_gpu_kv_shared_weights.py holds the kernels to, on the CPU: weights in two bf16 parts meet it;
where keys that hold less than a third of what is counted before them have one part, rows do not."""
import torch

import _kv_even_weights as E
import _kv_reference as R
import _kv_weights as W


def test_the_bound_tells_one_part_from_two():
    n, Hq, H, D, ctx = 40, 4, 2, 64, 1100
    K, V, Q = E.rows_on_eight_keys(n, ctx, 2, Hq, H, D, 5, "cpu")
    O, A, S, _ = W.exact(Q, K, V, torch.full((n,), ctx + 2))
    limit = W.bound(O, A, S, 0.0, ctx + 2)
    late = torch.arange(ctx + 2) % 64 >= 32
    for parts in (1, 2):
        got = torch.zeros_like(O)
        for h in range(Hq):
            z = Q[:, h].double() @ K[:, h // 2].double().T
            w = torch.exp(z - z.amax(1, keepdim=True) + 0.01)
            assert (w / w.sum(1, keepdim=True)).max() < 0.2
            assert (w[:, late].amax(1) < w[:, ~late].sum(1) / 3).all()
            top = R.bf16_of_f64(w).double()
            rest = R.bf16_of_f64(w - top).double()
            if parts == 1:
                rest[:, late] = 0
            got[:, h] = (top + rest) @ V[:, h // 2].double() / w.sum(1, keepdim=True)
        over = (R.bf16_of_f64(got).double() - O).abs() > limit
        assert over.any() == (parts == 1)
        if parts == 1:
            assert over.any(-1).double().mean() > 0.3
