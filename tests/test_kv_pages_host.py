"""The page tables' calls without a GPU: refusals come back before any device work; and the model that the
GPU tests compare with, on tables worked out by hand."""
import ctypes

import pytest
import torch

import adapter_linear_gb300 as al
from _kv_pages_reference import Tables
from adapter_linear_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def lib():
    if cuda_build.needs_build():
        cuda_build.build()
    return al.load_library()


def create(lib, pages=8, page=16, seqs=4, stride=4, table=64, kv_len=64, refs=64, out=True):
    h = ctypes.c_void_p()
    return lib.lora_kv_pages_create(pages, page, seqs, stride, table, kv_len, refs, ctypes.byref(h) if out else None)


def test_create_refuses_before_touching_the_device(lib):
    assert create(lib, out=False) == al.LORA_ERR_ARG
    for pages in (0, -1, (1 << 27) + 1):
        assert create(lib, pages=pages) == al.LORA_ERR_SHAPE
    for page in (0, 8, 24, 512):
        assert create(lib, page=page) == al.LORA_ERR_SHAPE
    for seqs in (0, 65537):
        assert create(lib, seqs=seqs) == al.LORA_ERR_SHAPE
    assert create(lib, stride=0) == al.LORA_ERR_SHAPE
    assert create(lib, stride=(1 << 26) + 1) == al.LORA_ERR_SHAPE            # 2^30 tokens and more
    assert create(lib, seqs=65536, stride=32768) == al.LORA_ERR_SHAPE        # 2^31 entries
    for name in ("table", "kv_len", "refs"):
        assert create(lib, **{name: None}) == al.LORA_ERR_ARG
        assert create(lib, **{name: 66}) == al.LORA_ERR_ARG


def test_null_handles(lib):
    n = ctypes.c_int()
    assert lib.lora_kv_pages_destroy(None) == al.LORA_ERR_ARG
    assert lib.lora_kv_pages_update(None, None, None, None, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_pages_compact(None, None, None, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_pages_used(None, ctypes.byref(n)) == al.LORA_ERR_ARG
    assert lib.lora_kv_pages_check_errors(None) == al.LORA_ERR_ARG
    assert lib.lora_kv_copy(None, None, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_copy_pages(None, 64, 64, None, 1, None) == al.LORA_ERR_ARG


def test_host_tensors_are_refused():
    for make in (lambda: al.KvPages(8, 16, 2, 4, device="cpu"),
                 lambda: al.KvPages(8, 16, 2, 4, tensors=(torch.zeros(2, 4, dtype=torch.int32),
                                                          torch.zeros(2, dtype=torch.int32),
                                                          torch.zeros(8, dtype=torch.int32)))):
        with pytest.raises(al.LoraError) as e:
            make()
        assert e.value.status == al.LORA_ERR_ARG
    with pytest.raises(al.LoraError) as e:
        al.KvPages(8, 16, 0, 4, device="cpu")
    assert e.value.status == al.LORA_ERR_SHAPE


@pytest.mark.parametrize("current", [0, 1])
def test_tensors_of_another_gpu_than_the_current_one_are_refused(current, monkeypatch):
    """(The handle belongs to the current GPU, the calls' streams to the tensors'.)"""
    from adapter_linear_gb300 import kv
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or al.LORA_OK

    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(kv, "load_library", Library)
    tensors = (torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32))
    if current == 1:
        al.KvPages(8, 16, 2, 4, tensors=tensors)
        assert calls == ["lora_kv_pages_create"]
        return
    with pytest.raises(al.LoraError) as e:
        al.KvPages(8, 16, 2, 4, tensors=tensors)
    assert e.value.status == al.LORA_ERR_ARG and calls == []


@pytest.mark.parametrize("current", [0, 1])
def test_arenas_on_another_gpu_than_the_current_one_are_refused(current, monkeypatch):
    from adapter_linear_gb300 import kv
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or al.LORA_OK

    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(kv, "load_library", Library)
    arenas = (*(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16) for _ in "kv"), None, None)
    if current == 1:
        al.KvCache(4, 16, 2, 64, al.LORA_KV_BF16, arenas=arenas)
        assert calls == ["lora_kv_create"]
        return
    with pytest.raises(al.LoraError) as e:
        al.KvCache(4, 16, 2, 64, al.LORA_KV_BF16, arenas=arenas)
    assert e.value.status == al.LORA_ERR_ARG and calls == []


def test_the_model():
    t = Tables(8, 16, 3, 4)
    assert t.update(room=[20, 16, 0]) == []
    assert t.table == [[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4] and t.len == [20, 16, 0]
    assert t.update(parent=[0, 1, 0], room=[0, 1, 0]) == [(1, 4, 4)]     # slot 1's new page comes first
    assert t.table == [[0, 1, -1, -1], [2, 3, -1, -1], [0, 4, -1, -1]] and t.refs() == [2, 1, 1, 1, 1, 0, 0, 0]
    assert t.update(parent=[-1, 2, 1]) == []
    assert t.table == [[-1] * 4, [0, 4, -1, -1], [2, 3, -1, -1]]
    assert t.compact() == [(4, 1, 16)] and t.table[1] == [0, 1, -1, -1]
    assert t.update(room=[0, 0, 48]) == "range" and t.update(room=[64, 16, 16]) == "oom"
