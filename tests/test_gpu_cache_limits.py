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


@pytest.mark.parametrize("D,dtype", [(64, torch.bfloat16), (80, torch.bfloat16), (64, torch.float32), (136, torch.float32)])
@pytest.mark.parametrize("back", [6, 40, 300])
def test_lengths_just_below_2_31(D, dtype, back):
    # the last positions that a table row can have, against the same keys and values near the start of another: the
    # tiles lie alike in both, so the results are equal bit for bit
    P, width, short, kmax, window, sinks = 32, (1 << 26) - 1, 41, 5, 500, 70
    far = width * P - back
    near = far - (width - short) * P   # a whole number of tiles before
    g = torch.Generator(device=DEV)
    g.manual_seed(back)
    k, v = (torch.randn((32, 2, P, D), generator=g, device=DEV).to(dtype) for _ in range(2))
    q = torch.randn((kmax + 1, 4, D), generator=g, device=DEV).to(dtype)
    order = torch.randperm(32, generator=g, device=DEV).to(torch.int32)
    got = []
    for n, pages in ((near, short), (far, width)):
        table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
        table[0, :3] = order[:3]
        table[0, pages - 27:pages] = order[3:30]
        length = torch.tensor([n], dtype=torch.int32, device=DEV)
        got.append(sv.spec_paged_attention(q, k, v, table, length, None, kmax, D ** -0.5, window=window, sinks=sinks))
    assert got[0]["status"].tolist() == [0] and got[1]["status"].tolist() == [0]
    assert torch.isfinite(got[1]["out"].float()).all()
    assert torch.equal(got[0]["out"], got[1]["out"])
    # and one token too many for the row
    length += back
    out = sv.spec_paged_attention(q, k, v, table, length, None, kmax, D ** -0.5, window=window, sinks=sinks)
    assert out["status"].tolist() == [9] and torch.isnan(out["out"].float()).all()
