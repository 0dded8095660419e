"""The decode loop of a target with rotary positions: a prompt that goes through whole decodes as one that goes through in blocks, prompts of several
streams at once as each alone, and speculation at temperature 0 emits what plain decoding emits."""

import pytest

import speculative_decoding_block_verify_gb300 as sv  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from speculative_decoding_block_verify_gb300 import decode_example as ex  # noqa: E402


def prompt(target, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(0, target.V, (n,), generator=g, device="cuda", dtype=torch.int32)


def greedy(target, cache, anchor, wanted, drafts):
    got, counts, status = ex.decode(torch, target, cache, anchor, wanted, drafts, torch.zeros(anchor.numel(), device="cuda"), target.table)
    assert (status == 0).all() and counts.min() >= 1
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_whole_and_blockwise_prompts_fill_the_same_cache(dtype):
    target = ex.Target(torch, rotary=True, dtype=dtype)
    tokens = prompt(target, 150, 1)
    caches = []
    for whole in (True, False):
        cache, state = ex.Cache(torch, target, 1, 400), {}
        if whole:
            ex.prefill_whole(torch, target, cache, tokens[:-1], [149], state)
            assert (state["status"] == 0).all()
        else:
            assert (ex.prefill(torch, target, cache, tokens, {}) == 0).all()
        assert cache.length.tolist() == [149]
        caches.append(cache)
    a, b = (torch.stack([c.k, c.v])[:, :, c.table[0, :9].long()].float() for c in caches)   # nine whole pages
    # The first layer's come from the same rows through products of other shapes.  A sum of 256 products is off by up to 256 u (u = 2^-24) of
    # |x| |w|, which is 16 on average where the largest of the sums is above 4: two are off by 2 2^-16 4 of that.  In bf16 each is rounded as well.
    assert (a[:, 0] - b[:, 0]).abs().max() <= (2.0 ** -7 if dtype == torch.bfloat16 else 0) * a[:, 0].abs().max() + 2.0 ** -13 * a[:, 0].abs().max()
    if dtype == torch.float32:
        assert torch.equal(greedy(target, caches[0], tokens[-1:], 24, 0), greedy(target, caches[1], tokens[-1:], 24, 0))


def test_several_prompts_at_once():
    target = ex.Target(torch, rotary=True)
    counts = [40, 0, 99, 1, 16]
    tokens = [prompt(target, n + 1, 10 + n) for n in counts]
    cache, state = ex.Cache(torch, target, len(counts), 300), {}
    logits = ex.prefill_whole(torch, target, cache, torch.cat([t[:-1] for t in tokens]), counts, state)
    assert logits.shape == (sum(counts), target.V) and (state["status"] == 0).all() and cache.length.tolist() == counts
    together = greedy(target, cache, torch.stack([t[-1] for t in tokens]), 16, 0)
    for b, n in enumerate(counts):
        cache = ex.Cache(torch, target, 1, 300)
        if n:
            ex.prefill_whole(torch, target, cache, tokens[b][:-1], [n], {})
        assert torch.equal(greedy(target, cache, tokens[b][-1:], 16, 0)[0], together[b])


def test_greedy_speculation_emits_what_plain_decoding_emits():
    target = ex.Target(torch, rotary=True)
    tokens = prompt(target, 77, 5)
    out = []
    for drafts in (0, 5):
        cache = ex.Cache(torch, target, 1, 400)
        ex.prefill_whole(torch, target, cache, tokens[:-1], [76], {})
        out.append(greedy(target, cache, tokens[-1:], 24, drafts)[0, :24])
    assert torch.equal(out[0], out[1])


def test_a_prompt_that_finds_no_page_keeps_nothing():
    target = ex.Target(torch, rotary=True)
    cache, state = ex.Cache(torch, target, 2, 64), {}
    cache.refs[3:] = 1   # three pages are left: the first prompt gets its two, the second none of its three
    ex.prefill_whole(torch, target, cache, prompt(target, 70, 6), [30, 40], state)
    assert state["status"].tolist() == [0, 8] and cache.length.tolist() == [30, 0]
