"""What spec_prompt_attention reports once a wait has given up.  The mark that such a wait leaves is set from the host: nothing waits here."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from speculative_decoding_block_verify_gb300 import decode_example as ex  # noqa: E402
from tests.test_gpu_prompt_attention import call, make  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TIMEOUT, BAD_OFFSETS = 6, 5


@pytest.fixture
def marked():
    sv.spec_prompt_mark_timeout(True)
    try:
        yield
    finally:
        sv.spec_prompt_mark_timeout()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,Hq,Hkv,D,window", [([40, 0, 300], 4, 2, 64, 0), ([700, 3], 4, 2, 64, 50), ([5] * 700, 2, 1, 128, 0), ([90], 2, 2, 256, 0)])
def test_every_prompt_reports_it_until_cleared(rows, Hq, Hkv, D, window, dtype):
    if dtype is F32 and D > 128:
        pytest.skip("refused")
    c = make(51, rows, Hq, Hkv, D, dtype)
    n = c["cu"][-1]
    want = call(c, window)["out"][:n].clone()
    sv.spec_prompt_mark_timeout(True)
    try:
        for _ in range(2):
            got = call(c, window)
            assert got["status"].tolist() == [TIMEOUT] * len(rows)
            assert torch.equal(got["out"][:n], want)   # nothing gave up: the rows are there
    finally:
        sv.spec_prompt_mark_timeout()
    got = call(c, window)
    assert got["status"].tolist() == [0] * len(rows) and torch.equal(got["out"][:n], want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broken_offsets_are_reported_first(dtype, marked):
    c = make(52, [5, 4, 3], 4, 2, 64, dtype, behind=0)
    c["d_cu"] = torch.tensor([0, 5, 4, 12], dtype=torch.int32, device="cuda")
    assert call(c)["status"].tolist() == [TIMEOUT, BAD_OFFSETS, BAD_OFFSETS]


def test_order_in_the_stream_and_in_a_graph():
    c = make(53, [30, 200], 4, 2, 64)
    before, after = call(c), call(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out=before)
        sv.spec_prompt_mark_timeout(True)
        call(c, out=after)
        sv.spec_prompt_mark_timeout(False)
    for _ in range(3):
        graph.replay()
        assert before["status"].tolist() == [0, 0] and after["status"].tolist() == [TIMEOUT] * 2
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_prompt_mark_timeout(True, stream=side)
    call(c, out=after, stream=side)
    sv.spec_prompt_mark_timeout(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert after["status"].tolist() == [TIMEOUT] * 2
    assert call(c)["status"].tolist() == [0, 0]


def test_a_prefill_that_timed_out_keeps_nothing(marked):
    target = ex.Target(torch, rotary=True)
    cache, state = ex.Cache(torch, target, 2, 64), {}
    ex.prefill_whole(torch, target, cache, torch.zeros(50, dtype=torch.int32, device="cuda"), [30, 20], state)
    assert state["status"].tolist() == [TIMEOUT] * 2 and cache.length.tolist() == [0, 0]
