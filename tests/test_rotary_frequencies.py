"""spec_rotary_frequencies against numbers worked out by hand, without any form of its formula (CPU only)."""

import ctypes
import math

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild

# a power is good to a few units in the last place, and a handful of roundings follow
CLOSE = dict(rtol=16 * 2.0 ** -52, atol=0)


def frequencies(dim, base, scaling=0, factor=1.0, original=4096.0, slow=1.0, fast=32.0):
    svbuild.build()
    f, m = (ctypes.c_double * (dim // 2))(), ctypes.c_float()
    assert sv.lib().spec_rotary_frequencies(dim, base, scaling, factor, original, slow, fast, f, ctypes.byref(m)) == 0
    return np.array(f), m.value


def test_plain_and_linear():
    f, m = frequencies(8, 10000.0)
    np.testing.assert_allclose(f, [1.0, 0.1, 0.01, 0.001], **CLOSE)
    assert m == 1.0
    np.testing.assert_allclose(frequencies(4, 9.0)[0], [1.0, 1 / 3], **CLOSE)
    np.testing.assert_allclose(frequencies(8, 10000.0, 1, 5.0)[0], [0.2, 0.02, 0.002, 0.0002], **CLOSE)


@pytest.mark.parametrize("dim", [4, 6, 64, 128])
def test_ntk_leaves_the_fastest_pair_and_stretches_the_slowest_by_the_factor(dim):
    plain, f = frequencies(dim, 10000.0)[0], frequencies(dim, 10000.0, 2, 8.0)[0]
    assert f[0] == 1.0
    np.testing.assert_allclose(f[-1], plain[-1] / 8, rtol=64 * 2.0 ** -52)
    # and those between by the same step from pair to pair
    np.testing.assert_allclose(f[1:] / f[:-1], np.full(dim // 2 - 1, f[1]), rtol=128 * 2.0 ** -52)


def test_yarn_by_turns_in_the_original_context():
    # 2,000 pi positions: the pairs turn 1,000, 100, 10 and 1 times; the border of slow 1 and fast 19 is half way at 10
    f, m = frequencies(8, 10000.0, 3, 4.0, 2000 * math.pi, 1.0, 19.0)
    np.testing.assert_allclose(f, [1.0, 0.1, 0.01 * (0.5 + 0.5 / 4), 0.001 / 4], rtol=64 * 2.0 ** -52)
    assert m == np.float32(1.0 + 0.1 * math.log(4.0))
    # all of them faster, all of them slower than the borders; a quarter of the way
    np.testing.assert_allclose(frequencies(8, 10000.0, 3, 4.0, 2000 * math.pi, 0.25, 0.5)[0], [1.0, 0.1, 0.01, 0.001], **CLOSE)
    np.testing.assert_allclose(frequencies(8, 10000.0, 3, 4.0, 2000 * math.pi, 2000.0, 3000.0)[0], [0.25, 0.025, 0.0025, 0.00025], **CLOSE)
    np.testing.assert_allclose(frequencies(8, 10000.0, 3, 4.0, 2000 * math.pi, 8.0, 16.0)[0][2], 0.01 * (0.25 + 0.75 / 4), rtol=64 * 2.0 ** -52)
    assert frequencies(64, 10000.0, 3, 1.0)[1] == 1.0
