"""The bounds of the float32 attention tests hold for the arithmetic that is meant, and fail without any piece of it (CPU only)."""

import numpy as np
import pytest

from tests import float32_parts as fp

N = 4096


@pytest.mark.parametrize("kind", ["scores", "weights"])
def test_the_whole_product_is_within_its_bound(kind):
    x = fp.two_key_inputs(kind, N, 1)
    want, bound = fp.two_key_output(*x)
    assert (np.abs(fp.two_key_model(*x) - want) <= bound).all()


@pytest.mark.parametrize("term", fp.TERMS)
def test_a_lost_term_is_noticed(term):
    x = fp.two_key_inputs("scores", N, 2)
    want, bound = fp.two_key_output(*x)
    assert (np.abs(fp.two_key_model(*x, without_scores=term) - want) > 2 * bound).any()
    x = fp.two_key_inputs("weights", N, 3)
    want, bound = fp.two_key_output(*x)
    assert (np.abs(fp.two_key_model(*x, without_values=term) - want) > 2 * bound).any()


@pytest.mark.parametrize("kind", ["scores", "weights"])
def test_two_parts_are_noticed(kind):
    x = fp.two_key_inputs(kind, N, 4)
    want, bound = fp.two_key_output(*x)
    assert (np.abs(fp.two_key_model(*x, n_parts=2) - want) > 2 * bound).any()


def test_the_shift_of_cut_sums_is_noticed():
    assert abs(fp.mean_shift(1, 200, 5003, 5)) <= fp.SHIFT
    assert abs(fp.mean_shift(79, 200, 5003, 5)) > 2 * fp.SHIFT
    assert fp.SHIFT < 5e-6
