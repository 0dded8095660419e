"""The decode loop over a pool that runs out of pages: a stream without a page waits, and nobody's tokens change."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from speculative_decoding_block_verify_gb300 import decode_example as ex  # noqa: E402


def run(pages, drafts, steps, streams=3, page=16, prompt_tokens=45):
    target = ex.Target(torch)
    cache = ex.Cache(torch, target, streams, 400, page=page, spare=pages - streams * 25)
    assert cache.refs.numel() == pages
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompt = torch.randint(0, target.V, (prompt_tokens,), generator=g, device="cuda", dtype=torch.int32)
    assert ex.prefill(torch, target, cache, prompt, {}).tolist() == [0]
    others = torch.arange(1, streams, dtype=torch.int32, device="cuda")
    assert (cache.fork(torch.zeros_like(others), others) == 0).all()
    # every stream goes on with a token of its own
    anchor = torch.arange(7, 7 + streams, dtype=torch.int32, device="cuda")
    got = ex.decode(torch, target, cache, anchor, steps, drafts, torch.zeros(streams, device="cuda"), target.table)
    return cache, got


@pytest.mark.parametrize("drafts", [0, 1, 5])
@pytest.mark.parametrize("pages", [4, 5, 7])
def test_streams_that_wait_emit_what_they_emit_with_room(drafts, pages):
    # 44 tokens are two full pages and 12 tokens of a third, shared by all three
    _, (plain, counts, status) = run(75, drafts, 24)
    assert (status == 0).all()
    cache, (got, counts, status) = run(pages, drafts, 24)
    waits = status != 0
    assert waits.any() and (counts[waits] == 0).all() and (counts[~waits] >= 1).all()
    assert set(status[waits].tolist()) == {8}
    n = counts.sum(dim=0).tolist()
    assert max(n) > 0
    assert torch.equal(cache.length.long(), 44 + counts.long().sum(dim=0))
    for b in range(3):
        both = min(n[b], int((plain[b] >= 0).sum()))
        assert torch.equal(got[b, :both], plain[b, :both]), b
        assert (got[b, n[b]:] == -1).all()


def test_a_prompt_that_does_not_fit_is_reported():
    target = ex.Target(torch)
    cache = ex.Cache(torch, target, 1, 400, page=16, spare=-23)
    prompt = torch.arange(50, dtype=torch.int32, device="cuda")
    assert ex.prefill(torch, target, cache, prompt, {}).tolist() == [8]
    assert int(cache.length[0]) == 0


def test_rows_that_are_too_short_are_refused_or_reported():
    target = ex.Target(torch, positions=64)
    cache = ex.Cache(torch, target, 2, 64, page=16)
    anchor, zero = torch.tensor([3, 4], dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError, match="68 tokens a stream"):
        ex.decode(torch, target, cache, anchor, 16, 3, zero, target.table)
    _, counts, status = ex.decode(torch, target, cache, anchor, 15, 3, zero, target.table)
    assert (status == 0).all() and torch.equal(cache.length.long(), counts.long().sum(dim=0))
    # a prompt longer than the row: nothing is read past the model's positions
    target = ex.Target(torch, positions=64)
    cache = ex.Cache(torch, target, 2, 64, page=16)
    prompt = torch.arange(101, dtype=torch.int32, device="cuda")
    assert ex.prefill(torch, target, cache, prompt, {}).tolist() == [9]
    assert cache.length.tolist() == [33, 0]
