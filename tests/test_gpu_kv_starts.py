"""Sequence starts that no caller should pass: reported, not followed, and the other sequences' rows
stay right."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

HIGH, LOW = 2 ** 31 - 1, -2 ** 31
# starts of the good batch [0, 3, 5, 7, 10], what is put in their place, the rows that stay right
STARTS = [
    ({2: HIGH, 3: LOW + 4}, range(0, 3)),         # the difference of the two wraps round to 5
    ({2: HIGH}, [0, 1, 2, 7, 8, 9]),
    ({2: -4}, [0, 1, 2, 7, 8, 9]),
    ({1: LOW}, range(5, 10)),
    ({0: HIGH}, range(3, 10)),
    ({0: -1}, range(3, 10)),
    ({4: 11}, range(0, 7)),
]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("case", range(len(STARTS)))
def test_bad_starts_are_not_followed(case, many):
    """many: 200 sequences of one token behind the four, so that the search takes two rounds."""
    bad, keep = STARTS[case]
    if many and 4 in bad:
        bad = {4: HIGH}
    more = 200 if many else 0
    lens, new = [100, 90, 80, 70] + [30] * more, [3, 2, 2, 3] + [1] * more
    p = R.Paged(al, al.LORA_KV_INT8, lens, new, 2, 128, 16, seed=160 + case)
    start = p.batch.start.clone()
    for i, v in bad.items():
        start[i] = v
    keep = torch.tensor(list(keep) + list(range(11, p.T)), device="cuda")
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    ref = R.attention(Q, p, 1.0 / math.sqrt(128))
    for max_new in (3, 40):                       # the short-chunk kernel alone, both kernels' walks
        batch = al.KvBatch(p.table, start, p.batch.kv_len, p.T, max_new)
        O, lse = p.cache.attention(Q, batch)
        assert p.cache.check_errors() == al.LORA_ERR_RANGE
        R.check_attention(O[keep], lse[keep], tuple(x[keep] for x in ref), f"{bad}")
    K, V = (torch.randn(p.T, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    p.cache.write(K, V, batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    Kr, Vr = p.cache.read(p.batch)                # with the good starts
    assert p.cache.check_errors() == al.LORA_OK
    Kb, Vb = p.cache.read(batch)
    assert p.cache.check_errors() == al.LORA_ERR_RANGE
    for x, got, again in ((K, Kr, Kb), (V, Vr, Vb)):
        q, s = R.quantise(x)
        want = R.bf16_of_f64(q * s[..., None])
        assert torch.equal(got[keep], want[keep]) and torch.equal(again[keep], want[keep])
