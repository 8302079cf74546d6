"""After a bounded wait has run out, which a test hook stands in for (nothing waits on the device),
check_errors reports it once and the cache's next calls are right."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
import _kv_reference as R

pytestmark = pytest.mark.gpu


# sequences split over CTAs, on the short-chunk kernel and on the tcgen05 one
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [70, 40]])
@pytest.mark.parametrize("fmt", [al.LORA_KV_INT8, al.LORA_KV_BF16])
def test_the_cache_works_again_after_a_timeout(fmt, new):
    p = R.Paged(al, fmt, [3000, 2500], new, 2, 128, 16, seed=220)
    Q = torch.randn(p.T, 8, 128, device="cuda").to(torch.bfloat16)
    p.cache.selftest_timeout()
    assert p.cache.check_errors() == al.LORA_ERR_TIMEOUT
    assert p.cache.check_errors() == al.LORA_OK
    ref = R.attention(Q, p, 1.0 / math.sqrt(128))
    for _ in range(3):
        O = torch.full_like(Q, float("nan"))
        lse = torch.full((p.T, 8), float("nan"), device="cuda")
        p.cache.attention(Q, p.batch, O=O, lse=lse)
        R.check_attention(O, lse, ref, f"{new}")
    assert p.cache.check_errors() == al.LORA_OK
