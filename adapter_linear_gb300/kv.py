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
from .rotary import Rotary


class _BatchStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("table_stride", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("T", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


class _GroupsStruct(ctypes.Structure):
    _fields_ = [("seq_start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p), ("n_groups", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32)]


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


class KvGroups:
    """Groups of a batch's sequences that share a prefix: sequences seq_start[g]..seq_start[g+1] hold the same
    first prefix_len[g] tokens, in the same pages as far as these are whole.

    seq_start int32 [n_groups + 1] and prefix_len int32 [n_groups] are device tensors (kept alive here, read
    when the kernels run), max_tokens a bound on the rows of one group."""

    def __init__(self, seq_start, prefix_len, max_tokens: int):
        for t in (seq_start, prefix_len):
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise LoraError(LORA_ERR_ARG, "KvGroups: seq_start and prefix_len are contiguous int32")
        n = prefix_len.shape[0]
        if seq_start.shape[0] != n + 1:
            raise LoraError(LORA_ERR_SHAPE, "KvGroups: seq_start has n_groups + 1 entries")
        self.device = seq_start.get_device()
        if self.device < 0 or prefix_len.get_device() != self.device:
            raise LoraError(LORA_ERR_ARG, "KvGroups: seq_start and prefix_len are on one GPU")
        self.tensors = (seq_start, prefix_len)
        self.struct = _GroupsStruct(seq_start.data_ptr(), prefix_len.data_ptr(), n, _clamped(max_tokens))
        self.ref = ctypes.byref(self.struct)


class KvCache:
    """A paged cache on the current GPU, of num_pages pages of page_tokens tokens for kv_heads heads of head_dim
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
        if self._device != torch._C._cuda_getDevice():  # (the handle would be the current one's)
            raise LoraError(LORA_ERR_ARG, "KvCache: the arenas are on the current GPU")
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

    def _empty_like(self, x, stream):
        """An output of x's shape, as _empty (torch takes 1 us less)."""
        if stream is None:
            return torch.empty_like(x, memory_format=torch.contiguous_format)
        with torch.cuda.stream(self._stream_object(stream)):
            return torch.empty_like(x, memory_format=torch.contiguous_format)

    def _empty(self, shape, dtype, stream):
        """An output, allocated for the stream that will write it."""
        if stream is None:  # (sizes one by one: a tuple takes torch 1 us more)
            return torch.empty(*shape, dtype=dtype, device=self._torch_device)
        with torch.cuda.stream(self._stream_object(stream)):
            return torch.empty(*shape, dtype=dtype, device=self._torch_device)

    def _rows(self, x, heads: int, batch: KvBatch, what: str) -> int:
        """The token stride of x, a bf16 [T, heads, head_dim] tensor with contiguous heads."""
        T, D = batch.T, self.head_dim
        if x.dtype is not torch.bfloat16 or x.shape != (T, heads, D):
            raise LoraError(LORA_ERR_SHAPE, f"{what}: bfloat16 [{T}, {heads}, {D}] expected")
        if x.get_device() != self._device or batch.device != self._device:
            raise LoraError(LORA_ERR_ARG, f"{what}: the tensors of a call are on the cache's GPU")
        if x.is_contiguous():
            return heads * D
        st, sh, sd = x.stride()
        if (sd != 1 and D > 1) or (sh != D and heads > 1):
            raise LoraError(LORA_ERR_ARG, f"{what}: the heads of a token must be contiguous")
        return st if T > 1 else heads * D

    def reserve(self, max_tokens: int, n_heads: int, max_seqs: int):
        _check(self._lib.lora_kv_reserve(self.handle, max_tokens, n_heads, max_seqs), "lora_kv_reserve")

    def write(self, K, V, batch: KvBatch, stream=None):
        """Write the batch's keys and values (bf16 [T, kv_heads, head_dim]) into their pages."""
        ks = self._rows(K, self.kv_heads, batch, "lora_kv_write K")
        vs = self._rows(V, self.kv_heads, batch, "lora_kv_write V")
        st = self._stream(stream, batch, K, V)
        _check(self._lib.lora_kv_write(self.handle, K.data_ptr(), ks, V.data_ptr(), vs, batch.ref, st),
               "lora_kv_write")

    def write_rotary(self, rotary: Rotary, K, V, batch: KvBatch, Q=None, Q_out=None, stream=None):
        """Write the batch's keys, rotated by their positions, and its values (as they are) into their pages. Q
        (bf16 [T, heads, head_dim]): rotated beside them into Q_out (Q itself: in place; by default a new
        tensor), which is returned."""
        what = "lora_kv_write_rotary"
        ks, vs = self._rows(K, self.kv_heads, batch, what + " K"), self._rows(V, self.kv_heads, batch, what + " V")
        qs = os_ = heads = 0
        if Q is not None:
            if Q.dim() != 3:
                raise LoraError(LORA_ERR_SHAPE, what + ": Q is [T, heads, head_dim]")
            heads = Q.shape[1]
            qs = self._rows(Q, heads, batch, what + " Q")
            if Q_out is None:
                Q_out = self._empty_like(Q, stream)
                os_ = heads * self.head_dim
            else:
                os_ = self._rows(Q_out, heads, batch, what + " Q_out")
        elif Q_out is not None:
            raise LoraError(LORA_ERR_ARG, what + ": Q_out without Q")
        st = self._stream(stream, batch, K, V, Q, Q_out)
        _check(self._lib.lora_kv_write_rotary(self.handle, rotary.ref, K.data_ptr(), ks, V.data_ptr(), vs, _ptr(Q), qs,
                                              heads, _ptr(Q_out), os_, batch.ref, st), what)
        return Q_out

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
        Q, qs, O, os_, lse, scale = self._attention_args("lora_kv_attention", Q, batch, scale, O, lse, stream)
        st = self._stream(stream, batch, Q, O, lse)
        _check(self._lib.lora_kv_attention(self.handle, Q.data_ptr(), qs, Q.shape[1], batch.ref, scale, _clamped(window),
                                           O.data_ptr(), os_, lse.data_ptr(), st), "lora_kv_attention")
        return O, lse

    def reserve_shared(self, max_tokens: int, n_heads: int, max_seqs: int):
        _check(self._lib.lora_kv_reserve_shared(self.handle, max_tokens, n_heads, max_seqs), "lora_kv_reserve_shared")

    def attention_shared(self, Q, batch: KvBatch, groups: Optional[KvGroups], scale: Optional[float] = None, O=None, lse=None,
                         stream=None):
        """attention() without a window, for a batch whose groups of sequences share prefixes (None: no groups):
        each group's prefix is read once, which pays for many short chunks over a long prefix."""
        Q, qs, O, os_, lse, scale = self._attention_args("lora_kv_attention_shared", Q, batch, scale, O, lse, stream)
        if groups is not None and groups.device != self._device:
            raise LoraError(LORA_ERR_ARG, "lora_kv_attention_shared: the tensors of a call are on the cache's GPU")
        st = self._stream(stream, batch, Q, O, lse, *(groups.tensors if groups is not None else ()))
        _check(self._lib.lora_kv_attention_shared(self.handle, Q.data_ptr(), qs, Q.shape[1], batch.ref,
                                                  groups.ref if groups is not None else None, scale,
                                                  O.data_ptr(), os_, lse.data_ptr(), st), "lora_kv_attention_shared")
        return O, lse

    def _attention_args(self, what, Q, batch, scale, O, lse, stream):
        if Q.dim() != 3:
            raise LoraError(LORA_ERR_SHAPE, f"{what}: Q is [T, n_heads, head_dim]")
        T, Hq, _ = Q.shape
        qs = self._rows(Q, Hq, batch, what + " Q")
        if O is None:
            O = self._empty_like(Q, stream)
            os_ = Hq * self.head_dim
        else:
            os_ = self._rows(O, Hq, batch, what + " O")
        if lse is None:
            lse = self._empty((T, Hq), torch.float32, stream)
        elif lse.dtype != torch.float32 or tuple(lse.shape) != (T, Hq) or not lse.is_contiguous():
            raise LoraError(LORA_ERR_SHAPE, f"{what} lse: contiguous float32 [T, n_heads] expected")
        elif lse.get_device() != self._device:
            raise LoraError(LORA_ERR_ARG, f"{what} lse: the tensors of a call are on the cache's GPU")
        return Q, qs, O, os_, lse, 1.0 / math.sqrt(self.head_dim) if scale is None else scale

    def copy(self, pages: "KvPages", stream=None):
        """Make the copies that the last update or compaction of `pages` asks for."""
        if pages._device != self._device:
            raise LoraError(LORA_ERR_ARG, "lora_kv_copy: the page tables are on the cache's GPU")
        st = self._stream(stream, pages)
        _check(self._lib.lora_kv_copy(self.handle, pages.handle, st), "lora_kv_copy")

    def copy_pages(self, src, dst, rows=None, stream=None):
        """Copy the first rows[i] (all) tokens of page src[i] to page dst[i] (int32 [n] tensors)."""
        lists = tuple(t for t in (src, dst, rows) if t is not None)
        for t in lists:
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.shape != src.shape:
                raise LoraError(LORA_ERR_SHAPE, "lora_kv_copy_pages: src, dst and rows are contiguous int32 [n]")
            if t.get_device() != self._device:
                raise LoraError(LORA_ERR_ARG, "lora_kv_copy_pages: the tensors of a call are on the cache's GPU")
        st = self._stream(stream, _Tensors(lists))
        _check(self._lib.lora_kv_copy_pages(self.handle, src.data_ptr(), dst.data_ptr(), _ptr(rows), src.shape[0], st),
               "lora_kv_copy_pages")

    def check_errors(self) -> int:
        return self._lib.lora_kv_check_errors(self.handle)

    def selftest_timeout(self, stream=None):
        """Test hook: leaves the cache as calls do whose bounded waits ran out."""
        _check(self._lib.lora_kv_selftest_timeout(self.handle, self._stream(stream)), "lora_kv_selftest_timeout")


class _Tensors:
    """Tensors a call uses, where a KvBatch stands otherwise."""

    def __init__(self, tensors):
        self.tensors = tensors


class KvPages:
    """The page tables of max_seqs sequences over num_pages pages of page_tokens tokens: `table` int32 [max_seqs,
    max_entries], `kv_len` int32 [max_seqs] and `refs` int32 [num_pages] (table entries that name a page),
    tensors on the current GPU that a KvBatch may name. tensors: (table, kv_len, refs) to use in place of new, empty ones.

    Calls run on the current stream or on `stream`. They change the tables; KvCache.copy then makes the copies
    they ask for, in each cache."""

    def __init__(self, num_pages: int, page_tokens: int, max_seqs: int, max_entries: int, device="cuda",
                 tensors: Optional[Tuple] = None):
        self.handle = None
        self.num_pages, self.page_tokens, self.max_seqs, self.max_entries = num_pages, page_tokens, max_seqs, max_entries
        if tensors is None:
            if min(num_pages, max_seqs, max_entries) < 1:
                raise LoraError(LORA_ERR_SHAPE, "KvPages: num_pages, max_seqs and max_entries are positive")
            table = torch.full((max_seqs, max_entries), -1, dtype=torch.int32, device=device)
            kv_len, refs = (torch.zeros(n, dtype=torch.int32, device=device) for n in (max_seqs, num_pages))
        else:
            table, kv_len, refs = tensors
        self._device = table.get_device()
        self._state(table, refs, "KvPages")
        self._slots(kv_len, "KvPages: kv_len")
        if self._device != torch._C._cuda_getDevice():  # (the handle would be the current one's)
            raise LoraError(LORA_ERR_ARG, "KvPages: the tensors are on the current GPU")
        self.table, self.kv_len, self.refs = table, kv_len, refs
        self.tensors = (table, kv_len, refs)
        h = ctypes.c_void_p()
        self._lib = load_library()
        _check(self._lib.lora_kv_pages_create(num_pages, page_tokens, max_seqs, max_entries, table.data_ptr(),
                                              kv_len.data_ptr(), refs.data_ptr(), ctypes.byref(h)),
               "lora_kv_pages_create")
        self.handle = h.value

    def close(self):
        if self.handle:
            self._lib.lora_kv_pages_destroy(self.handle)
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

    def _state(self, table, refs, what):
        for t, shape in ((table, (self.max_seqs, self.max_entries)), (refs, (self.num_pages,))):
            if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
                raise LoraError(LORA_ERR_SHAPE, f"{what}: contiguous int32 {shape} expected")
            if self._device < 0 or t.get_device() != self._device:
                raise LoraError(LORA_ERR_ARG, f"{what}: the tensors are on one GPU")

    def _slots(self, t, what):
        if t.dtype != torch.int32 or tuple(t.shape) != (self.max_seqs,) or not t.is_contiguous():
            raise LoraError(LORA_ERR_SHAPE, f"{what} is contiguous int32 [{self.max_seqs}]")
        if self._device < 0 or t.get_device() != self._device:
            raise LoraError(LORA_ERR_ARG, f"{what} is on the tables' GPU")

    def _stream(self, stream, *tensors) -> int:
        current = torch._C._cuda_getCurrentRawStream(self._device)
        if stream is None:
            return current
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        if handle != current:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, self.table.device)
            for t in tensors + self.tensors:
                if t is not None:
                    t.record_stream(stream)
        return handle

    def update(self, parent=None, keep=None, room=None, stream=None):
        """Slot i becomes the first keep[i] tokens (all) of what slot parent[i] (itself) holds, -1: nothing, and
        room[i] (0) tokens behind them; int32 [max_seqs] tensors. Follow it with KvCache.copy in each cache
        unless every slot keeps its own tokens."""
        for t, name in ((parent, "parent"), (keep, "keep"), (room, "room")):
            if t is not None:
                self._slots(t, f"lora_kv_pages_update: {name}")
        st = self._stream(stream, parent, keep, room)
        _check(self._lib.lora_kv_pages_update(self.handle, _ptr(parent), _ptr(keep), _ptr(room), st),
               "lora_kv_pages_update")

    def compact(self, out: Optional[Tuple] = None, stream=None):
        """Number the used pages from 0. out: (table, refs) for the new state, by default this object's own. Follow
        it with KvCache.copy in each cache."""
        table, refs = out if out is not None else (None, None)
        if out is not None:
            self._state(table, refs, "lora_kv_pages_compact")
        st = self._stream(stream, table, refs)
        _check(self._lib.lora_kv_pages_compact(self.handle, _ptr(table), _ptr(refs), st), "lora_kv_pages_compact")

    def used(self) -> int:
        """Pages in use, once the calls so far are done."""
        n = ctypes.c_int(0)
        _check(self._lib.lora_kv_pages_used(self.handle, ctypes.byref(n)), "lora_kv_pages_used")
        return n.value

    def check_errors(self) -> int:
        return self._lib.lora_kv_pages_check_errors(self.handle)
