"""Binding of the paged key/value cache and the attention over it (``include/lora_kv.h``).

``KvCache`` owns the arenas (torch tensors) and the handle; ``KvBatch`` names the tokens of
one step. As in the rest of the package every operator runs in the CUDA library, there is no
fall-back, and a refusal is a ``LoraError`` with the library's status.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import LORA_ERR_ARG, LORA_ERR_SHAPE, LORA_KV_BF16, LORA_KV_INT8, LoraError, _check, _ptr, load_library


class _BatchStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("table_stride", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("T", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


def _clamped(x: int) -> int:
    """x as the library's int takes it: ctypes would drop high bits; above 2^30 nothing differs, and
    any negative number is refused."""
    return max(-1, min(x, 1 << 30))


class KvBatch:
    """The tokens of one step: rows start[b]..start[b+1] of the step's tensors are the last
    tokens of sequence b, whose kv_len[b] tokens lie in the pages page_table[b] names.

    page_table int32 [n_seqs, entries], start int32 [n_seqs + 1] and kv_len int32 [n_seqs] are
    device tensors (kept alive here, read when the kernels run); T is the number of rows of
    the step's tensors and max_new a bound on the rows of one sequence."""

    def __init__(self, page_table, start, kv_len, T: int, max_new: int):
        for t, nd in ((page_table, 2), (start, 1), (kv_len, 1)):
            if t.dtype != torch.int32 or t.dim() != nd or not t.is_contiguous():
                raise LoraError(LORA_ERR_ARG, "KvBatch: page_table, start and kv_len are contiguous int32")
        self.device = page_table.get_device()
        if self.device < 0 or start.get_device() != self.device or kv_len.get_device() != self.device:
            raise LoraError(LORA_ERR_ARG, "KvBatch: page_table, start and kv_len are on one GPU")
        n = page_table.shape[0]
        if start.shape[0] != n + 1 or kv_len.shape[0] != n:
            raise LoraError(LORA_ERR_SHAPE, "KvBatch: start has n_seqs + 1 entries, kv_len n_seqs")
        self.page_table, self.start, self.kv_len, self.T = page_table, start, kv_len, T
        self.tensors = (page_table, start, kv_len)
        self.struct = _BatchStruct(page_table.data_ptr(), start.data_ptr(), kv_len.data_ptr(),
                                   page_table.shape[1], n, T, _clamped(max_new))
        self.ref = ctypes.byref(self.struct)


class KvCache:
    """A paged cache of num_pages pages of page_tokens tokens for kv_heads heads of head_dim
    values, bf16 or int8 with a bf16 scale per row. arenas: the tensors (k, v, k_scales,
    v_scales; the scales None for bf16) to use in place of newly allocated ones.

    Calls run on the current stream or on `stream` (a torch stream or a handle), which then has to
    follow what filled their inputs; outputs that a call allocates belong to the stream it runs on."""

    def __init__(self, num_pages: int, page_tokens: int, kv_heads: int, head_dim: int, fmt: int = LORA_KV_INT8,
                 device="cuda", arenas: Optional[Tuple] = None):
        self.handle = None
        self.num_pages, self.page_tokens = num_pages, page_tokens
        self.kv_heads, self.head_dim, self.fmt = kv_heads, head_dim, fmt
        shape = (num_pages, kv_heads, page_tokens, head_dim)
        dtype = torch.int8 if fmt == LORA_KV_INT8 else torch.bfloat16
        if arenas is None:
            k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
            ks, vs = ((torch.zeros(shape[:3], dtype=torch.bfloat16, device=device) for _ in range(2))
                      if fmt == LORA_KV_INT8 else (None, None))
        else:
            k, v, ks, vs = arenas
        for t in (k, v):
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
                raise LoraError(LORA_ERR_SHAPE, f"KvCache: pages are contiguous {shape} of {dtype}")
        for t in (ks, vs):
            if t is not None and (tuple(t.shape) != shape[:3] or t.dtype != torch.bfloat16 or
                                  not t.is_contiguous()):
                raise LoraError(LORA_ERR_SHAPE, f"KvCache: scales are contiguous {shape[:3]} of bfloat16")
        self._torch_device, self._device = k.device, k.get_device()
        if self._device < 0 or any(t is not None and t.get_device() != self._device for t in (v, ks, vs)):
            raise LoraError(LORA_ERR_ARG, "KvCache: the arenas are on one GPU")
        self.k, self.v, self.k_scales, self.v_scales = k, v, ks, vs
        h = ctypes.c_void_p()
        _check(load_library().lora_kv_create(num_pages, page_tokens, kv_heads, head_dim, fmt, _ptr(k), _ptr(v),
                                             _ptr(ks), _ptr(vs), ctypes.byref(h)), "lora_kv_create")
        self.handle = h.value
        self._lib = load_library()

    def close(self):
        if self.handle:
            self._lib.lora_kv_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001
            pass

    def _stream(self, stream, batch=None, *tensors) -> int:
        """The handle to launch on. On a stream other than the current one the allocator learns that
        it uses the call's tensors."""
        current = torch._C._cuda_getCurrentRawStream(self._device)  # (current_stream() builds an object: 3 us)
        if stream is None:
            return current
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        if handle != current and batch is not None:
            stream = self._stream_object(stream)
            for t in tensors + batch.tensors + (self.k, self.v, self.k_scales, self.v_scales):
                if t is not None:
                    t.record_stream(stream)
        return handle

    def _stream_object(self, stream):
        return torch.cuda.ExternalStream(stream, self._torch_device) if isinstance(stream, int) else stream

    def _empty(self, shape, dtype, stream):
        """An output, allocated for the stream that will write it."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._torch_device)
        with torch.cuda.stream(self._stream_object(stream)):
            return torch.empty(shape, dtype=dtype, device=self._torch_device)

    def _rows(self, x, heads: int, batch: KvBatch, what: str) -> int:
        """The token stride of x, a bf16 [T, heads, head_dim] tensor with contiguous heads."""
        T, D = batch.T, self.head_dim
        if x.dtype != torch.bfloat16 or x.dim() != 3 or x.shape[0] != T or x.shape[1] != heads or x.shape[2] != D:
            raise LoraError(LORA_ERR_SHAPE, f"{what}: bfloat16 [{T}, {heads}, {D}] expected")
        if x.get_device() != self._device or batch.device != self._device:
            raise LoraError(LORA_ERR_ARG, f"{what}: the tensors of a call are on the cache's GPU")
        s = x.stride()
        if (s[2] != 1 and D > 1) or (s[1] != D and heads > 1):
            raise LoraError(LORA_ERR_ARG, f"{what}: the heads of a token must be contiguous")
        return s[0] if T > 1 else heads * D

    def reserve(self, max_tokens: int, n_heads: int, max_seqs: int):
        _check(self._lib.lora_kv_reserve(self.handle, max_tokens, n_heads, max_seqs), "lora_kv_reserve")

    def write(self, K, V, batch: KvBatch, stream=None):
        """Write the batch's keys and values (bf16 [T, kv_heads, head_dim]) into their pages."""
        ks = self._rows(K, self.kv_heads, batch, "lora_kv_write K")
        vs = self._rows(V, self.kv_heads, batch, "lora_kv_write V")
        st = self._stream(stream, batch, K, V)
        _check(self._lib.lora_kv_write(self.handle, K.data_ptr(), ks, V.data_ptr(), vs, batch.ref, st),
               "lora_kv_write")

    def read(self, batch: KvBatch, K=None, V=None, stream=None):
        """The batch's tokens as bf16 [T, kv_heads, head_dim] keys and values."""
        shape = (batch.T, self.kv_heads, self.head_dim)
        if batch.device != self._device:
            raise LoraError(LORA_ERR_ARG, "lora_kv_read: the tensors of a call are on the cache's GPU")
        ks = vs = self.kv_heads * self.head_dim
        if K is None:
            K = self._empty(shape, torch.bfloat16, stream)
        else:
            ks = self._rows(K, self.kv_heads, batch, "lora_kv_read K")
        if V is None:
            V = self._empty(shape, torch.bfloat16, stream)
        else:
            vs = self._rows(V, self.kv_heads, batch, "lora_kv_read V")
        st = self._stream(stream, batch, K, V)
        _check(self._lib.lora_kv_read(self.handle, K.data_ptr(), ks, V.data_ptr(), vs, batch.ref, st),
               "lora_kv_read")
        return K, V

    def attention(self, Q, batch: KvBatch, scale: Optional[float] = None, window: int = 0, O=None, lse=None,
                  stream=None):
        """Attention of the batch's tokens over the cache, which already holds them.
        Q bf16 [T, n_heads, head_dim]; returns O (as Q) and lse fp32 [T, n_heads]."""
        if Q.dim() != 3:
            raise LoraError(LORA_ERR_SHAPE, "lora_kv_attention: Q is [T, n_heads, head_dim]")
        T, Hq, _ = Q.shape
        qs = self._rows(Q, Hq, batch, "lora_kv_attention Q")
        if O is None:
            O = self._empty((T, Hq, self.head_dim), torch.bfloat16, stream)
            os_ = Hq * self.head_dim
        else:
            os_ = self._rows(O, Hq, batch, "lora_kv_attention O")
        if lse is None:
            lse = self._empty((T, Hq), torch.float32, stream)
        elif lse.dtype != torch.float32 or tuple(lse.shape) != (T, Hq) or not lse.is_contiguous():
            raise LoraError(LORA_ERR_SHAPE, "lora_kv_attention lse: contiguous float32 [T, n_heads] expected")
        elif lse.get_device() != self._device:
            raise LoraError(LORA_ERR_ARG, "lora_kv_attention lse: the tensors of a call are on the cache's GPU")
        if scale is None:
            scale = 1.0 / math.sqrt(self.head_dim)
        st = self._stream(stream, batch, Q, O, lse)
        _check(self._lib.lora_kv_attention(self.handle, Q.data_ptr(), qs, Hq, batch.ref, scale, _clamped(window),
                                           O.data_ptr(), os_, lse.data_ptr(), st), "lora_kv_attention")
        return O, lse

    def check_errors(self) -> int:
        return self._lib.lora_kv_check_errors(self.handle)

    def selftest_timeout(self, stream=None):
        """Test hook: leaves the cache as calls do whose bounded waits ran out."""
        _check(self._lib.lora_kv_selftest_timeout(self.handle, self._stream(stream)), "lora_kv_selftest_timeout")
