"""Host-side checks of the paged cache's calls (no GPU): every refusal comes back before any
device work, as a status."""
import ctypes

import pytest

import adapter_linear_gb300 as al
from adapter_linear_gb300 import build as cuda_build
from adapter_linear_gb300.kv import _BatchStruct


@pytest.fixture(scope="module")
def lib():
    if cuda_build.needs_build():
        cuda_build.build()
    return al.load_library()


def create(lib, pages=4, page=16, heads=2, dim=64, fmt=al.LORA_KV_INT8, k=64, v=64, ks=64, vs=64, out=True):
    h = ctypes.c_void_p()
    return lib.lora_kv_create(pages, page, heads, dim, fmt, k, v, ks, vs, ctypes.byref(h) if out else None)


def test_create_refuses_before_touching_the_device(lib):
    assert create(lib, out=False) == al.LORA_ERR_ARG
    assert create(lib, fmt=2) == al.LORA_ERR_ARG
    for page in (0, 8, 24, 512, -16):
        assert create(lib, page=page) == al.LORA_ERR_SHAPE
    for dim in (0, 32, 96, 256):
        assert create(lib, dim=dim) == al.LORA_ERR_SHAPE
    for heads in (0, 257, -1):
        assert create(lib, heads=heads) == al.LORA_ERR_SHAPE
    assert create(lib, pages=0) == al.LORA_ERR_SHAPE
    assert create(lib, pages=1 << 30) == al.LORA_ERR_SHAPE          # 2^31 cache rows and more
    assert create(lib, k=None) == al.LORA_ERR_ARG
    assert create(lib, v=72) == al.LORA_ERR_ARG                     # alignment
    assert create(lib, ks=None) == al.LORA_ERR_ARG                  # int8 needs scales
    assert create(lib, fmt=al.LORA_KV_BF16) == al.LORA_ERR_ARG      # bf16 takes none


def test_null_handles(lib):
    b = ctypes.byref(_BatchStruct(64, 64, 64, 1, 1, 1, 1))
    assert lib.lora_kv_destroy(None) == al.LORA_ERR_ARG
    assert lib.lora_kv_reserve(None, 1, 1, 1) == al.LORA_ERR_ARG
    assert lib.lora_kv_write(None, 64, 128, 64, 128, b, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_read(None, 64, 128, 64, 128, b, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_attention(None, 64, 128, 2, b, 1.0, 0, 64, 128, None, None) == al.LORA_ERR_ARG
    assert lib.lora_kv_check_errors(None) == al.LORA_ERR_ARG
