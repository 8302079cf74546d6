"""What the binding of the paged cache refuses or hands on by itself (no GPU)."""
import math

import pytest
import torch

import adapter_linear_gb300 as al
from adapter_linear_gb300.kv import KvBatch, KvCache, _BatchStruct


def refused(status, call):
    with pytest.raises(al.LoraError) as e:
        call()
    assert e.value.status == status


def ints(*values):
    return torch.tensor(values, dtype=torch.int32)


class FakeLibrary:
    """Records what the library would be called with."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or al.LORA_OK


def a_cache_on(device_index):
    """A cache whose tensors claim to be on GPU device_index, without one."""
    c = KvCache.__new__(KvCache)
    c.handle, c._device, c.kv_heads, c.head_dim = None, device_index, 2, 64
    c._lib = FakeLibrary()
    return c


def a_batch_on(device_index, T):
    b = KvBatch.__new__(KvBatch)
    b.device, b.T, b.tensors, b.ref = device_index, T, (), None
    return b


def test_host_tensors_are_refused():
    refused(al.LORA_ERR_ARG, lambda: KvBatch(ints(0, 1).view(1, 2), ints(0, 1), ints(5), 1, 1))
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    refused(al.LORA_ERR_ARG, lambda: KvCache(4, 16, 2, 64, al.LORA_KV_BF16, arenas=(k, k.clone(), None, None)))
    refused(al.LORA_ERR_ARG, lambda: KvCache(4, 16, 2, 64, al.LORA_KV_INT8, device="cpu"))
    c, b = a_cache_on(0), a_batch_on(0, 3)
    K, Q = (torch.zeros(3, h, 64, dtype=torch.bfloat16) for h in (2, 4))
    refused(al.LORA_ERR_ARG, lambda: c.write(K, K, b))
    refused(al.LORA_ERR_ARG, lambda: c.read(b, K=K, V=K))
    refused(al.LORA_ERR_ARG, lambda: c.attention(Q, b))
    assert c._lib.calls == []


def test_tensors_of_another_device_are_refused():
    c, b = a_cache_on(-1), a_batch_on(1, 3)       # -1: what the host's tensors answer
    K, Q = (torch.zeros(3, h, 64, dtype=torch.bfloat16) for h in (2, 4))
    refused(al.LORA_ERR_ARG, lambda: c.write(K, K, b))
    refused(al.LORA_ERR_ARG, lambda: c.read(b))
    refused(al.LORA_ERR_ARG, lambda: c.attention(Q, b))
    assert c._lib.calls == []


@pytest.mark.parametrize("window,given", [(0, 0), (5, 5), (2 ** 31, 2 ** 30), (2 ** 32 + 5, 2 ** 30), (-1, -1),
                                          (-2 ** 32, -1)])
def test_no_window_loses_its_high_bits(window, given, monkeypatch):
    c, b = a_cache_on(-1), a_batch_on(-1, 3)
    monkeypatch.setattr(KvCache, "_stream", lambda self, stream, *args: 0)
    Q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    c.attention(Q, b, window=window, O=torch.zeros_like(Q), lse=torch.zeros(3, 4))
    (name, args), = c._lib.calls
    assert name == "lora_kv_attention" and args[6] == given and args[5] == 1 / math.sqrt(64)


def test_a_bound_on_the_rows_loses_no_high_bits():
    from adapter_linear_gb300.kv import _clamped
    for max_new, kept in ((3, 3), (2 ** 32, 2 ** 30), (-2 ** 32 + 1, -1)):
        assert _BatchStruct(0, 0, 0, 1, 1, 1, _clamped(max_new)).max_new == kept
