"""Rotary positions without a GPU: the frequencies of every scaling, the fixed-point steps, refusals."""
import ctypes
import fractions
import math

import pytest
import torch

import adapter_linear_gb300 as al
from adapter_linear_gb300 import build as cuda_build
from adapter_linear_gb300.rotary import Rotary, _RotaryStruct


@pytest.fixture(scope="module", autouse=True)
def lib():
    if cuda_build.needs_build():
        cuda_build.build()
    return al.load_library()


def refused(status, call):
    with pytest.raises(al.LoraError) as e:
        call()
    assert e.value.status == status


def plain_frequencies(R, base, kind, scale, trained, options):
    """freq and factor from the definitions, pair by pair."""
    out, factor = [], 1.0
    if kind == "ntk":
        base *= scale ** (R / (R - 2))
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        turns = trained * f / (2 * math.pi)
        if kind == "linear":
            f /= scale
        if kind == "bands":
            near = min(1, max(0, (turns - options[0]) / (options[1] - options[0])))
            f = near * f + (1 - near) * f / scale
        if kind == "yarn":
            def pair(n):
                return R * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(pair(options[0]))), min(R - 1, math.ceil(pair(options[1])))
            far = min(1, max(0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f = far * f / scale + (1 - far) * f
            factor = 0.1 * math.log(scale) + 1 if scale > 1 else 1.0
        out.append(f)
    return out, factor


@pytest.mark.parametrize("R", [16, 64, 96, 128, 256])
@pytest.mark.parametrize("kind,options", [(None, None), ("linear", None), ("ntk", None), ("yarn", (32.0, 1.0)),
                                          ("yarn", (8.0, 2.0)), ("bands", (1.0, 4.0)), ("bands", (0.5, 30.0))])
@pytest.mark.parametrize("base,scale,trained", [(10000.0, 8.0, 8192), (500000.0, 40.0, 4096), (1e6, 1.0, 1000)])
def test_frequencies(R, kind, options, base, scale, trained):
    r = Rotary(R, base, scaling=None if kind is None else (kind, scale, trained), options=options)
    want, factor = plain_frequencies(R, base, kind, scale, trained, options)
    # pow, log and a handful of fp64 operations, a few 2^-53 each; the ends of yarn's ramp are whole numbers
    # here (no logarithm falls within 2^-40 of one)
    assert r.factor == pytest.approx(factor, rel=2.0 ** -48)
    assert r.freq == pytest.approx(want, rel=2.0 ** -44)


def test_steps_are_the_frequencies_in_turns():
    freq = [1.0, 2 * math.pi, -0.25, 1e-7, 100.0, 0.0, 3.0, 6.283185]
    r = Rotary(16, freq=freq, factor=2.0)
    for f, step in zip(freq, r.struct.step):
        turns = f / (2 * math.pi)
        got = step / 2.0 ** 64
        # fp64's rounding of the quotient and of its fraction
        assert abs((got - turns + 0.5) % 1.0 - 0.5) <= 2.0 ** -52 * max(1.0, abs(turns))
    assert list(r.struct.step[8:]) == [0] * 120 and r.struct.factor == 2.0


def test_negative_frequencies_turn_back_as_far():
    freq = [0.25, 1e-3, 1e-7, 1e-12, 3.0, 2 * math.pi, 7.5, 1.0]
    there, back = (Rotary(16, freq=[sign * f for f in freq]).struct.step[:8] for sign in (1, -1))
    assert [(a + b) % 2 ** 64 for a, b in zip(there, back)] == [0] * 8
    # against pi to 40 digits: the quotient's rounding and 2 pi's, 2^-52 of it together, and what 2^-64 cuts off
    two_pi = 2 * fractions.Fraction("3.1415926535897932384626433832795028841972")
    for f, step in zip(freq, back):
        turns = fractions.Fraction(f) / two_pi
        off = (fractions.Fraction(step, 2 ** 64) + turns) % 1
        assert min(off, 1 - off) <= turns / 2 ** 52 + fractions.Fraction(1, 2 ** 64), f


def test_refusals(lib):
    refused(al.LORA_ERR_SHAPE, lambda: Rotary(24))
    refused(al.LORA_ERR_SHAPE, lambda: Rotary(0))
    refused(al.LORA_ERR_SHAPE, lambda: Rotary(272))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, layout="other"))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, scaling=("other", 2.0, 100)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, base=0.0))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, base=float("nan")))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, scaling=("linear", -1.0, 100)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, scaling=("bands", 2.0, 0)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, scaling=("bands", 2.0, 100), options=(4.0, 4.0)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, scaling=("yarn", 2.0, 100), options=(1.0, 32.0)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, base=1.0, scaling=("yarn", 2.0, 100)))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, freq=[1.0] * 15))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, freq=[1.0] * 15 + [float("inf")]))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32, factor=float("inf")))
    f = (ctypes.c_double * 16)()
    assert lib.lora_rotary_frequencies(32, 1e4, 0, 1.0, 1.0, None, None, None) == al.LORA_ERR_ARG
    assert lib.lora_rotary_frequencies(32, 1e4, 7, 1.0, 1.0, None, f, f) == al.LORA_ERR_ARG
    assert lib.lora_rotary_init(32, 2, f, 1.0, ctypes.byref(_RotaryStruct())) == al.LORA_ERR_ARG
    assert lib.lora_rotary_init(32, 0, None, 1.0, ctypes.byref(_RotaryStruct())) == al.LORA_ERR_ARG


def test_apply_refuses_before_touching_the_device(lib):
    from adapter_linear_gb300.rotary import _TENSORS
    r = Rotary(32)

    def call(n=1, head_dim=64, pos=64, T=3, rot=None, inp=64, out=128, stride=128, out_stride=128, heads=2):
        arr = _TENSORS[1].pack(inp or 0, out or 0, stride, out_stride, heads, 0) * 5
        return lib.lora_rotary_apply(rot or r.ref, n, arr, head_dim, pos, T, 0, None)

    for n in (0, 5):
        assert call(n=n) == al.LORA_ERR_ARG
    for d in (16, 40, 272):
        assert call(head_dim=d) == al.LORA_ERR_SHAPE
    assert call(T=-1) == al.LORA_ERR_ARG
    assert call(pos=None) == al.LORA_ERR_ARG and call(pos=66) == al.LORA_ERR_ARG
    assert call(inp=None) == al.LORA_ERR_ARG and call(out=None) == al.LORA_ERR_ARG
    assert call(inp=72) == al.LORA_ERR_ARG and call(out=72) == al.LORA_ERR_ARG
    assert call(stride=120) == al.LORA_ERR_ARG and call(out_stride=132) == al.LORA_ERR_ARG
    assert call(heads=0) == al.LORA_ERR_ARG
    assert call(out=64, out_stride=256) == al.LORA_ERR_ARG           # in place with two strides
    bad = _RotaryStruct()
    assert call(rot=ctypes.byref(bad)) == al.LORA_ERR_ARG             # never initialised
    assert call(T=0, pos=None) == al.LORA_OK
    assert lib.lora_kv_write_rotary(None, r.ref, 64, 128, 64, 128, None, 0, 0, None, 0, None, None) == al.LORA_ERR_ARG


def test_host_tensors_are_refused():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    refused(al.LORA_ERR_ARG, lambda: Rotary(32).apply((x,), pos))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32).apply((), pos))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32).apply((x,) * 5, pos))
    refused(al.LORA_ERR_ARG, lambda: Rotary(32).apply((x,), pos.long()))
    refused(al.LORA_ERR_SHAPE, lambda: Rotary(32).apply((x.float(),), pos))
    refused(al.LORA_ERR_SHAPE, lambda: Rotary(32).apply((x[:2],), pos))
