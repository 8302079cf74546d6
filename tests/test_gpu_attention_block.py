"""The example block: LoRA projections, cache, attention and o_proj together, prefill to decode."""
import os
import sys

import pytest

import adapter_linear_gb300 as al

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bound", [(al.LORA_KV_BF16, 0.02), (al.LORA_KV_INT8, 0.03)])
def test_prefill_chunks_and_decode_agree_with_the_plain_block(fmt, bound):
    """Bounds on a token's relative error: five roundings to bf16 on the way (projection, cache,
    weights, attention's output, o_proj: 2^-8 each at most, so 2 % even if they all add up), and
    8-bit rows, off by up to half a step of amax / 127 (uniform: 0.23 % of amax, amax about
    3 standard deviations: 0.7 %), in K and in V."""
    import lora_attention_block as ex
    assert ex.run(fmt) <= bound
