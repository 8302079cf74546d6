"""Binding of rotary positions (``include/lora_rotary.h``).

``Rotary`` is a rotation: its frequencies, layout and factor, plain host memory. ``Rotary.apply`` rotates
tensors of tokens; ``KvCache.write_rotary`` rotates keys on their way into the cache and queries beside them.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence, Tuple

import torch

from . import LORA_ERR_ARG, LORA_ERR_SHAPE, LoraError, _check, load_library

LORA_ROTARY_MAX_DIM = 256
LORA_ROTARY_MAX_TENSORS = 4
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class _RotaryStruct(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("factor", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("step", ctypes.c_uint64 * (LORA_ROTARY_MAX_DIM // 2))]


# n lora_rotary_tensor in a row: two addresses, two strides, heads, reserved
_TENSORS = [struct.Struct("PPqqii" * n) for n in range(LORA_ROTARY_MAX_TENSORS + 1)]


class Rotary:
    """The rotation of the first rotary_dim values of a head (a multiple of 16), pairs by `layout`:
    "half" (i, i + rotary_dim / 2) or "interleaved" (2 i, 2 i + 1).

    Frequencies are base^(-2 i / rotary_dim), changed by scaling: None, or (kind, scale, trained) with kind
    "linear", "ntk", "yarn" or "bands" for `scale` times the context of `trained` tokens the model was trained
    for (options: the kind's two bounds in turns); or freq, rotary_dim / 2 numbers of one's own. factor
    multiplies the result (by default what the scaling gives)."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: Optional[Tuple] = None, options: Optional[Sequence[float]] = None,
                 freq: Optional[Sequence[float]] = None, factor: Optional[float] = None):
        kind, scale, trained = scaling if scaling is not None else (None, 1.0, 1.0)
        if layout not in LAYOUTS or kind not in SCALINGS:
            raise LoraError(LORA_ERR_ARG, f"Rotary: layout is one of {sorted(LAYOUTS)}, scaling (kind, scale, trained) "
                                          f"with a kind of {sorted(k for k in SCALINGS if k)}")
        if rotary_dim < 16 or rotary_dim > LORA_ROTARY_MAX_DIM or rotary_dim % 16:
            raise LoraError(LORA_ERR_SHAPE, "Rotary: rotary_dim is a multiple of 16 up to 256")
        lib, n = load_library(), rotary_dim // 2
        f, own_factor = (ctypes.c_double * n)(), ctypes.c_double(1.0)
        if freq is not None:
            if len(freq) != n or scaling is not None:
                raise LoraError(LORA_ERR_ARG, "Rotary: freq is rotary_dim / 2 numbers, in place of a scaling")
            f[:] = [float(x) for x in freq]
        else:
            o = (ctypes.c_double * 2)(*options) if options is not None else None
            _check(lib.lora_rotary_frequencies(rotary_dim, base, SCALINGS[kind], scale, trained, o, f,
                                               ctypes.byref(own_factor)), "lora_rotary_frequencies")
        self.rotary_dim, self.layout = rotary_dim, layout
        self.factor = own_factor.value if factor is None else factor
        self.freq = list(f)
        self.struct = _RotaryStruct()
        self.ref = ctypes.byref(self.struct)
        _check(lib.lora_rotary_init(rotary_dim, LAYOUTS[layout], f, self.factor, self.ref), "lora_rotary_init")
        self._lib = lib

    def apply(self, tensors, positions, out=None, inverse: bool = False, stream=None):
        """Rotate up to four bf16 tensors [T, heads, head_dim] of the same tokens, at positions (int32 [T]).

        Heads of a token are contiguous, tokens may be strided. out: tensors for the results (those of
        `tensors` themselves: in place); by default new ones, returned as a tuple. inverse: the other
        way round (the gradient). Runs on the current stream or on `stream`."""
        if positions.dtype is not torch.int32 or positions.dim() != 1 or not positions.is_contiguous():
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: positions are contiguous int32 [T]")
        xs = tensors if type(tensors) is tuple else tuple(tensors)
        n, device, T = len(xs), positions.get_device(), positions.shape[0]
        if not 1 <= n <= LORA_ROTARY_MAX_TENSORS or (out is not None and len(out) != n):
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: one to four tensors, as many results")
        D = xs[0].shape[-1]
        given = [self._rows(x, None, T, D, device) for x in xs]
        if device < 0 or device != torch._C._cuda_getDevice():
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the tensors are on the current GPU")
        handle, other = torch._C._cuda_getCurrentRawStream(device), None
        if stream is not None:
            where = stream if isinstance(stream, int) else stream.cuda_stream
            if where != handle:
                other = torch.cuda.ExternalStream(stream, positions.device) if isinstance(stream, int) else stream
            handle = where
        fields, results = [], []
        for i, x in enumerate(xs):
            stride, heads = given[i]
            if out is not None:
                y = out[i]
                to_stride, _ = self._rows(y, heads, T, D, device)
            else:
                if other is None:
                    y = torch.empty_like(x, memory_format=torch.contiguous_format)
                else:
                    with torch.cuda.stream(other):  # it belongs to the stream that writes it
                        y = torch.empty_like(x, memory_format=torch.contiguous_format)
                to_stride = heads * D
            results.append(y)
            fields += (x.data_ptr(), y.data_ptr(), stride, to_stride, heads, 0)
        if other is not None:
            for t in (*xs, *results, positions):
                t.record_stream(other)
        _check(self._lib.lora_rotary_apply(self.ref, n, _TENSORS[n].pack(*fields), D, positions.data_ptr(), T, inverse,
                                           handle), "lora_rotary_apply")
        return tuple(results)

    @staticmethod
    def _rows(x, heads, T, D, device):
        """Token stride and heads of x, a bf16 [T, heads, D] tensor with contiguous heads."""
        if x.dtype is not torch.bfloat16 or x.dim() != 3:
            raise LoraError(LORA_ERR_SHAPE, f"lora_rotary_apply: bfloat16 [{T}, heads, {D}] expected")
        t, h, d = x.shape
        if t != T or d != D or (heads is not None and h != heads):
            raise LoraError(LORA_ERR_SHAPE, f"lora_rotary_apply: bfloat16 [{T}, {heads or 'heads'}, {D}] expected")
        if x.get_device() != device:
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the tensors of a call are on one GPU")
        if x.is_contiguous():
            return h * D, h
        st, sh, sd = x.stride()
        if (sd != 1 and D > 1) or (sh != D and h > 1):
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the heads of a token must be contiguous")
        return st if T > 1 else h * D, h
