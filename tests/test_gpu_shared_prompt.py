"""The shared-prompt example: rotary write, page tables, copies and shared attention together, as one served
block would use them. Bounds on a token's relative error: six roundings to bf16 on the way (projection,
rotated queries, cache, weights, attention's output, o_proj: 2^-8 each at most, 2.35 % if they all add up),
and with 8-bit rows up to half a step of amax / 127 in K and in V (uniform: 0.7 % each), 3 % taken."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
al = pytest.importorskip("adapter_linear_gb300")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt,bound", [(al.LORA_KV_INT8, 0.03), (al.LORA_KV_BF16, 0.0235)])
@pytest.mark.parametrize("prompts,answers", [((70, 129), 4), ((16, 1, 200), 3), ((33,), 16)])
def test_shared_prompt(fmt, bound, prompts, answers):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lora_shared_prompt
    assert lora_shared_prompt.run(fmt, prompts, answers) <= bound
