"""The cache calls at the ends of the sizes that they accept."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


def test_more_pages_asked_for_than_32_bits_count():
    # nine streams ask for 2^28 - 1 pages each (together above 2^31), the one behind them for a single one
    B, width, pages = 11, (1 << 28) - 1, 40
    k = torch.zeros((1, pages, 1, 8, 8), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    held, length, refs = i32(B), i32(B), i32(pages)
    room = torch.tensor([24] + [width * 8] * 9 + [8], dtype=torch.int32, device=DEV)
    out = sv.spec_cache_resize(k, k.clone(), table, held, length, refs, room=room)
    assert out["status"].tolist() == [0] + [8] * 10
    assert held.tolist() == [3] + [0] * 10
    assert refs.tolist() == [1] * 3 + [0] * 37
    assert table[:, :4].tolist() == [[0, 1, 2, -1]] + [[-1] * 4] * 10
