"""RotaryTable with frequencies of the caller's own (CPU only)."""

import math

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild


@pytest.fixture(scope="module", autouse=True)
def library():
    svbuild.build()


@pytest.mark.parametrize("scaling,factor,want", [("yarn", 16.0, 0.1 * math.log(16.0) + 1), ("yarn", 1.0, 1.0), ("none", 1.0, 1.0), ("linear", 8.0, 1.0),
                                                 ("ntk", 8.0, 1.0), ("linear", 0.5, 1.0)])
def test_magnitude_beside_given_frequencies(scaling, factor, want):
    f = [0.5 ** j for j in range(32)]
    t = sv.RotaryTable(64, scaling=scaling, factor=factor, frequencies=f, device="cpu")
    assert t.magnitude == np.float32(want)
    assert t.frequencies == f   # as they are given
    assert sv.RotaryTable(64, scaling=scaling, factor=factor, frequencies=f, magnitude=1.5, device="cpu").magnitude == 1.5


def test_refused_beside_given_frequencies():
    for kw in [dict(scaling="yarn", factor=0.5), dict(scaling="yarn", factor=math.nan), dict(scaling="other")]:
        with pytest.raises((ValueError, sv.SpecError)):
            sv.RotaryTable(64, frequencies=[0.5] * 32, device="cpu", **kw)
    # a magnitude of one's own asks nothing of the factor
    assert sv.RotaryTable(64, frequencies=[0.5] * 32, device="cpu", scaling="yarn", factor=0.5, magnitude=1.0).magnitude == 1.0
