"""The mark of a prompt attention's wait that gave up: refusals before any launch (CPU only)."""

import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild


@pytest.mark.parametrize("marked", [2, -1, 256])
def test_marks_are_0_or_1(marked):
    svbuild.build()
    assert sv.lib().spec_prompt_mark_timeout(marked, None) == -1
    assert b"marked" in sv.lib().spec_last_error()
