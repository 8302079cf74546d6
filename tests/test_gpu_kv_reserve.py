"""After lora_kv_reserve an attention call of that size allocates nothing: it can be captured in a graph
(where an allocation fails)."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu

# Hq, H, lens, new, max_new given (None: exact)
CASES = [
    (32, 1, [300, 40, 7], [1, 1, 1], None),          # single tokens, 32 heads on one kv head
    (8, 1, [300, 40, 7, 90], [4, 0, 0, 0], None),    # as many tokens as sequences, of one sequence
    (64, 1, [200], [1], None),
    (8, 2, [300, 40, 7], [1, 1, 1], 1000),           # a loose bound
    (8, 8, [300, 40], [1, 1], 64),
]


@pytest.mark.parametrize("fmt", [al.LORA_KV_INT8, al.LORA_KV_BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_reserved_call_can_be_captured(case, fmt):
    Hq, H, lens, new, bound = CASES[case]
    p = R.Paged(al, fmt, lens, new, H, 128, 16, seed=190 + case)
    n = len(lens)
    assert p.T <= n
    batch = al.KvBatch(p.table, p.batch.start, p.batch.kv_len, p.T, max(new) if bound is None else bound)
    p.cache.reserve(p.T, Hq, n)
    Q = torch.randn(p.T, Hq, 128, device="cuda").to(torch.bfloat16)
    O, lse = torch.zeros_like(Q), torch.zeros(p.T, Hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.cache.attention(Q, batch, O=O, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    R.check_attention(O, lse, R.attention(Q, p, 1.0 / math.sqrt(128)), f"{CASES[case]}")
    assert p.cache.check_errors() == al.LORA_OK
