"""Sizes of the cache calls that are refused on the host (CPU only)."""

import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild
from tests.test_cache_abi import P, append, attention


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


def test_pages_times_heads_is_a_coordinate(L):
    # bf16 pages are copied by (page, head) number, a 32-bit coordinate; one past the last one stands for "no page"
    for pages, Hkv, dtype, code in [(1 << 30, 2, 1, -3), ((1 << 31) - 1, 1, 1, -3), (1 << 30, 2, 0, -6), ((1 << 30) - 1, 2, 1, -6)]:
        args = attention(pages=pages, Hkv=Hkv, Hq=8, dtype=dtype, ws=0)
        rc = L.spec_paged_attention(args, None)
        # without a device the call that passes the sizes' checks ends at the device's attributes
        assert rc == code or (code == -6 and rc == -4), (pages, Hkv, dtype, rc)


def test_append_reserved_errors(L):
    assert L.spec_cache_append_reserved(None, None, None) == -1
    assert L.spec_cache_append_reserved(append(), None, None) == -1
    assert b"reserved" in L.spec_last_error()
    for change, code in [(dict(dtype=-1), -2), (dict(kmax=33), -3), (dict(page=20), -3), (dict(rows=-1), -3), (dict(kp=0), -1)]:
        assert L.spec_cache_append_reserved(append(**change), P, None) == code, change
    assert L.spec_cache_append_reserved(append(B=0), None, None) == 0


def test_scales_that_overflow_to_base_2(L):
    for scale, ok in [(2.3e38, True), (2.5e38, False), (-3.4e38, False), (-2.3e38, True)]:
        rc = L.spec_paged_attention(attention(scale=scale, ws=0), None)
        assert (rc in (-4, -6)) if ok else rc == -1, (scale, rc)
