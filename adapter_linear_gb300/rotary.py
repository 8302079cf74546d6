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
        xs = tuple(tensors)
        n = len(xs)
        if not 1 <= n <= LORA_ROTARY_MAX_TENSORS:
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: one to four tensors")
        if positions.dtype != torch.int32 or positions.dim() != 1 or not positions.is_contiguous():
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: positions are contiguous int32 [T]")
        T, D, device = positions.shape[0], xs[0].shape[-1], positions.get_device()
        given = [self._rows(x, None, T, D, device) for x in xs]
        if device < 0 or device != torch._C._cuda_getDevice():
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the tensors are on the current GPU")
        handle = current = torch._C._cuda_getCurrentRawStream(device)
        other = None
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            if handle != current:
                other = torch.cuda.ExternalStream(stream, xs[0].device) if isinstance(stream, int) else stream
        if out is None:
            if other is None:
                out = tuple([torch.empty_like(x, memory_format=torch.contiguous_format) for x in xs])
            else:
                with torch.cuda.stream(other):  # they belong to the stream that writes them
                    out = tuple([torch.empty_like(x, memory_format=torch.contiguous_format) for x in xs])
            results = [(y.data_ptr(), h * D, h) for y, (_, _, h) in zip(out, given)]
        else:
            out = tuple(out)
            if len(out) != n:
                raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: as many results as tensors")
            results = [self._rows(y, h, T, D, device) for y, (_, _, h) in zip(out, given)]
        fields = []
        for (a, sa, h), (b, sb, _) in zip(given, results):
            fields += (a, b, sa, sb, h, 0)
        if other is not None:
            for t in xs + out + (positions,):
                t.record_stream(other)
        _check(self._lib.lora_rotary_apply(self.ref, n, _TENSORS[n].pack(*fields), D, positions.data_ptr(), T, inverse,
                                           handle), "lora_rotary_apply")
        return out

    @staticmethod
    def _rows(x, heads, T, D, device):
        """Address, token stride and heads of x, a bf16 [T, heads, D] tensor with contiguous heads."""
        if x.dim() != 3 or x.dtype != torch.bfloat16:
            raise LoraError(LORA_ERR_SHAPE, f"lora_rotary_apply: bfloat16 [{T}, heads, {D}] expected")
        t, h, d = x.shape
        if t != T or d != D or (heads is not None and h != heads):
            raise LoraError(LORA_ERR_SHAPE, f"lora_rotary_apply: bfloat16 [{T}, {heads or 'heads'}, {D}] expected")
        if x.get_device() != device:
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the tensors of a call are on one GPU")
        st, sh, sd = x.stride()
        if (sd != 1 and D > 1) or (sh != D and h > 1):
            raise LoraError(LORA_ERR_ARG, "lora_rotary_apply: the heads of a token must be contiguous")
        return x.data_ptr(), st if T > 1 else h * D, h
