"""The decode loop: speculative decoding at temperature 0 emits what plain decoding emits, whatever the drafts are;
forked streams decode as streams that were prefilled themselves; pages are never lost."""

import pytest

import speculative_decoding_block_verify_gb300 as sv  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from speculative_decoding_block_verify_gb300 import decode_example as ex  # noqa: E402


def setup(streams, prompt_tokens, tokens, page=16, **kw):
    target = ex.Target(torch, **kw)
    cache = ex.Cache(torch, target, streams, tokens, page=page)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompt = torch.randint(0, target.V, (prompt_tokens,), generator=g, device="cuda", dtype=torch.int32)
    ex.prefill(torch, target, cache, prompt, {})
    if streams > 1:
        others = torch.arange(1, streams, dtype=torch.int32, device="cuda")
        assert (cache.fork(torch.zeros_like(others), others) == 0).all()
    return target, cache, prompt, target.table


@pytest.mark.parametrize("page,prompt", [(8, 45), (16, 64), (64, 101)])
def test_greedy_speculation_emits_what_plain_decoding_emits(page, prompt):
    B, wanted = 3, 24
    zero = torch.zeros(B, device="cuda")
    target, cache, tokens, drafter = setup(B, prompt, 400, page=page)
    plain, counts, status = ex.decode(torch, target, cache, tokens[-1:].repeat(B), wanted, 0, zero, drafter)
    assert (status == 0).all() and (counts == 1).all()
    assert (plain[0] == plain[1]).all() and (plain[0] == plain[2]).all()   # forked streams are the prompt's
    for drafts in (1, 5):
        target, cache, tokens, drafter = setup(B, prompt, 400, page=page)
        got, counts, status = ex.decode(torch, target, cache, tokens[-1:].repeat(B), wanted, drafts, zero, drafter)
        assert (status == 0).all() and counts.min() >= 1
        assert counts.float().mean() > 1.1   # drafts are accepted, so blocks of several tokens are kept
        n = int(counts.sum(dim=0).min())
        n = min(n, wanted)
        assert torch.equal(got[:, :n], plain[:, :n])


def test_sampled_streams_hold_their_pages_alone():
    B, drafts, steps = 6, 4, 12
    target, cache, tokens, drafter = setup(B, 70, 300, dtype=torch.bfloat16)
    T = torch.full((B,), 0.9, device="cuda")
    got, counts, status = ex.decode(torch, target, cache, tokens[-1:].repeat(B), steps, drafts, T, drafter, seed=7)
    assert (status == 0).all()
    assert torch.equal(cache.length.long(), 69 + counts.long().sum(dim=0))
    held = torch.zeros_like(cache.refs)
    for b in range(B):
        row = cache.table[b][:int(cache.held[b])].long()
        held.index_add_(0, row, torch.ones_like(row, dtype=torch.int32))
        # the page that is being written into is the stream's own
        assert int(cache.refs[cache.table[b][int(cache.length[b]) // cache.page].long()]) == 1
    assert torch.equal(held, cache.refs)
    assert len({tuple(r) for r in got[:, :8].tolist()}) > 1   # streams have uniforms of their own
    cache.resize(advance=-cache.length)
    assert int(cache.refs.sum()) == 0
