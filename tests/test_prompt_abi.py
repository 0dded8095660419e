"""The prompt calls' host side: argument structs as the C compiler lays them out, errors that are answered before any launch,
frequencies and turns (CPU only)."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild
from tests import prompt_reference as ref


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


P = 4096   # a pointer that is never followed: the checks come first


def prompt(**kw):
    a = dict(B=2, Hq=8, Hkv=2, D=64, dtype=1, window=0, sinks=0, scale=0.125, rows=12, cu=P, q=P, k=P, v=P, qs=512, ks=128, vs=128, out=P,
             status=P)
    a.update(kw)
    return sv._PROMPT.pack(*a.values())


def rotate(**kw):
    a = dict(heads=8, D=64, dim=64, inter=0, dtype=1, mag=1.0, rows=12, turns=P, at=P, x=P, xs=512, out=P + 512, os=512)
    a.update(kw)
    return sv._ROTATE.pack(*a.values())


def append(**kw):
    a = dict(B=2, most=6, extra=1, Hq=8, Hkv=2, D=64, page=16, pages=100, width=10, dtype=1, dim=64, inter=0, mag=1.0, turns=P, cu=P, length=P,
             table=P, reserved=0, q=P, k=P, v=P, qs=512, ks=128, vs=128, rows=12, qo=P + 512, ko=P + 512, qos=512, kos=128, kp=P, vp=P, status=P)
    a.update(kw)
    return sv._APPEND_ROTATED.pack(*a.values())


def test_struct_sizes():
    assert (sv._PROMPT.size, sv._ROTATE.size, sv._APPEND_ROTATED.size) == (112, 80, 208)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), -2), (dict(B=-1), -3), (dict(B=65536), -3), (dict(Hq=9), -3), (dict(Hkv=0), -3), (dict(Hq=129, Hkv=1, qs=129 * 64), -3),
    (dict(D=60), -3), (dict(D=264), -3), (dict(D=0), -3), (dict(dtype=0, D=136, qs=2000, ks=2000, vs=2000), -3), (dict(window=-1), -3), (dict(sinks=-1), -3),
    (dict(qs=511), -3), (dict(ks=127), -3), (dict(vs=0), -3), (dict(rows=-1), -3), (dict(rows=1 << 31), -3), (dict(cu=0, rows=11), -3),
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(out=0), -1), (dict(status=0), -1), (dict(q=P + 2), -1), (dict(k=P + 8), -1),
    (dict(v=P + 4), -1), (dict(out=P + 8), -1), (dict(qs=513), -1), (dict(ks=132), -1), (dict(dtype=0, vs=130), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(scale=3e38), -1)])
def test_prompt_errors(L, change, code):
    assert L.spec_prompt_attention(prompt(**change), None) == code
    assert L.spec_last_error() != b""


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -2), (dict(heads=0), -3), (dict(heads=4097), -3), (dict(D=60), -3), (dict(D=264), -3), (dict(dim=0), -3), (dict(dim=63), -3),
    (dict(dim=66), -3), (dict(rows=-1), -3), (dict(rows=1 << 31), -3), (dict(xs=511), -3), (dict(os=511), -3), (dict(out=P, os=520), -3), (dict(mag=math.inf), -1),
    (dict(turns=0), -1), (dict(turns=P + 4), -1), (dict(at=0), -1), (dict(x=0), -1), (dict(out=0), -1)])
def test_rotate_errors(L, change, code):
    assert L.spec_rotate(rotate(**change), None) == code
    assert L.spec_last_error() != b""


@pytest.mark.parametrize("change,code", [
    (dict(dtype=-1), -2), (dict(B=-1), -3), (dict(B=65536), -3), (dict(most=-1), -3), (dict(extra=2), -3), (dict(extra=-1), -3), (dict(Hq=-1), -3),
    (dict(Hq=1025, qs=1 << 20, qos=1 << 20), -3), (dict(Hkv=0), -3), (dict(D=12), -3), (dict(dim=66), -3), (dict(dim=1), -3), (dict(page=20), -3), (dict(page=512), -3),
    (dict(pages=0), -3), (dict(width=0), -3), (dict(width=1 << 28), -3), (dict(qs=511), -3), (dict(ks=127), -3), (dict(vs=127), -3), (dict(qos=511), -3),
    (dict(kos=127), -3), (dict(qo=P, qos=520), -3), (dict(ko=P, kos=136), -3), (dict(rows=-1), -3), (dict(rows=1 << 31), -3), (dict(cu=0, rows=11), -3),
    (dict(mag=math.nan), -1), (dict(turns=0), -1), (dict(turns=P + 2), -1), (dict(length=0), -1), (dict(table=0), -1), (dict(q=0), -1), (dict(qo=0), -1), (dict(k=0), -1),
    (dict(v=0), -1), (dict(kp=0), -1), (dict(vp=P + 8), -1), (dict(status=0), -1)])
def test_append_errors(L, change, code):
    assert L.spec_cache_append_rotated(append(**change), None) == code
    assert L.spec_last_error() != b""


def test_nothing_to_do(L):
    for f in (L.spec_prompt_attention, L.spec_rotate, L.spec_cache_append_rotated):
        assert f(None, None) == -1
    assert L.spec_prompt_attention(prompt(B=0), None) == 0
    assert L.spec_rotate(rotate(rows=0, x=0, out=0, at=0), None) == 0
    assert L.spec_cache_append_rotated(append(B=0), None) == 0
    assert L.spec_last_error() == b""


def frequencies(L, dim, base=10000.0, scaling=0, factor=1.0, original=4096, slow=1.0, fast=32.0):
    f, m = (ctypes.c_double * (dim // 2))(), ctypes.c_float()
    rc = L.spec_rotary_frequencies(dim, base, scaling, factor, original, slow, fast, f, ctypes.byref(m))
    return rc, list(f), m.value


@pytest.mark.parametrize("dim", [2, 4, 20, 64, 80, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_frequencies(L, dim, scaling):
    for base, factor, original in [(10000.0, 1.0, 4096), (500000.0, 8.0, 8192), (1000000.0, 3.5, 32768)]:
        rc, f, m = frequencies(L, dim, base, sv.RotaryTable.SCALINGS[scaling], factor, original)
        assert rc == 0
        want = ref.frequencies(dim, base, scaling, factor, original)
        # a power of a rounded exponent (2^-53 of up to ln(base') = 30), and a few roundings
        assert np.abs(np.array(f) / want - 1).max() <= 40 * 2.0 ** -53
        assert m == (np.float32(0.1 * math.log(factor) + 1) if scaling == "yarn" else 1.0)


def test_frequency_errors(L):
    for kw in [dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5),
               dict(scaling=2, factor=math.nan), dict(scaling=3, original=0), dict(scaling=3, slow=32.0), dict(scaling=3, fast=math.inf)]:
        assert frequencies(L, 64, **kw)[0] == -1, kw
    for dim in (0, 1, 63, 258):
        f, m = (ctypes.c_double * 200)(), ctypes.c_float()
        assert L.spec_rotary_frequencies(dim, 1e4, 0, 1.0, 1.0, 1.0, 32.0, f, ctypes.byref(m)) == -3
    one = (ctypes.c_double * 1)(math.inf)
    t = (ctypes.c_uint64 * 1)()
    assert L.spec_rotary_turns(one, 1, t) == -1 and L.spec_rotary_turns(None, 1, t) == -1 and L.spec_rotary_turns(one, 0, t) == -3
    assert L.spec_rotary_turns(one, 129, t) == -3


def test_turns(L):
    # 2 pi to 200 bits
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    f = [1.0, 0.5, 1e-6, 3.0, 6.283185307179586, 7.0, -1.0, 0.0, 12345.678, 2.0 ** -60]
    t = (ctypes.c_uint64 * len(f))()
    assert L.spec_rotary_turns((ctypes.c_double * len(f))(*f), len(f), t) == 0
    for x, got in zip(f, t):
        want = Fraction(x) / two_pi
        off = (Fraction(got, 2 ** 64) - want) % 1
        off = min(off, 1 - off)
        # the division and 2 pi are rounded to 2^-53 of the quotient, taking the whole turns off leaves 2^-54 at most, the last step 2^-65
        assert off <= abs(want) * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 54), (x, float(off))


def test_table_checks(L):
    for kw in [dict(scaling="other"), dict(frequencies=[1.0]), dict(base=0.5)]:
        with pytest.raises((ValueError, sv.SpecError)):
            sv.RotaryTable(64, device="cpu", **kw)
    with pytest.raises(ValueError):
        sv.RotaryTable(63, device="cpu")
    t = sv.RotaryTable(64, frequencies=[0.25] * 32, magnitude=2, device="cpu")
    assert t.magnitude == 2.0 and t.frequencies == [0.25] * 32 and t.turns.shape == (32,)
