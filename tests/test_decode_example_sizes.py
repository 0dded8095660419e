"""The decode example's model has as many positions as its cache (the host's check, CPU only)."""

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_block_verify_gb300 import decode_example as ex  # noqa: E402


def test_a_cache_longer_than_the_model_is_refused():
    target = ex.Target(torch, V=8, width=8, layers=1, q_heads=1, kv_heads=1, head=8, positions=64, device="cpu")
    cache = ex.Cache(torch, target, 1, 65, device="cpu")
    with pytest.raises(ValueError, match="80 tokens a stream, the model for 64"):
        ex.forward(torch, target, cache, torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0, {})
