"""A prompt's way into the paged cache and on into decoding, with the calls that a layer makes, against the whole of it in 64 bits."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import prompt_reference as ref  # noqa: E402

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prompts_then_blocks(dtype, window, sinks):
    Hq, Hkv, D, P, N, steps = 8, 2, 64, 16, 3, 4
    prompts = [1, 100, 0, 333, 64]
    B, total = len(prompts), [p + steps * (N + 1) for p in prompts]
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    # every stream's projections of its whole life
    life = [torch.randn((n, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype) for n in total]
    t = sv.RotaryTable(D, scaling="yarn", factor=4.0, original=128)
    f, m = ref.frequencies(D, scaling="yarn", factor=4.0, original=128), 0.1 * np.log(4.0) + 1
    width, pages = 40, B * 40
    pool = [torch.full((1, pages, Hkv, P, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    table, held, length, refs = i32([[-1] * width] * B), i32([0] * B), i32([0] * B), i32([0] * pages)
    book = (table, held, length, refs)
    want = []
    for x in life:
        at = torch.arange(x.shape[0], device=DEV)
        q, k = sv.spec_rotate(x[:, :Hq], at.int(), t), sv.spec_rotate(x[:, Hq:Hq + Hkv], at.int(), t)
        for got, raw in ((q, x[:, :Hq]), (k, x[:, Hq:Hq + Hkv])):
            y, tol = ref.rotate(raw, at, f, m)
            assert ((got.double() - y).abs() <= tol).all()
        out, spread = ref.attention(q, k, x[:, Hq + Hkv:], [0, x.shape[0]], D ** -0.5, window, sinks)
        want.append((out, ref.attention_tolerance(q, k, D ** -0.5, x.shape[0], out, spread) if x.shape[0] else out))
    # the prompts: room, append, attention over the packed rows, tokens kept
    status = sv.spec_cache_resize(*pool, *book, room=i32(prompts))["status"]
    x = torch.cat([life[b][:prompts[b]] for b in range(B)])
    cu = i32([0] + list(np.cumsum(prompts)))
    a = sv.spec_cache_append_rotated(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pool[0][0], pool[1][0], table, length, t, cu_rows=cu, keep_keys=True,
                                     reserved=status)
    o = sv.spec_prompt_attention(a["q"], a["k"], x[:, Hq + Hkv:], cu, D ** -0.5, window, sinks)
    assert (a["status"] == 0).all() and (o["status"] == 0).all()
    r = 0
    for b in range(B):
        w, tol = want[b]
        n = prompts[b]
        assert ((o["out"][r:r + n].double() - w[:n]).abs() <= tol[:n]).all(), b
        r += n
    sv.spec_cache_resize(*pool, *book, advance=i32(prompts), room=i32([N + 1] * B))
    assert length.tolist() == prompts
    # the last token of a prompt again, as a block of one over the pages: the same row
    back = i32([-1 if p else 0 for p in prompts])
    for b in (1, 3, 4):
        last = x[int(cu[b + 1]) - 1:int(cu[b + 1])]
        q = sv.spec_rotate(last[:, :Hq], length[b:b + 1] - 1, t)
        got = sv.spec_paged_attention(q, pool[0][0], pool[1][0], table[b:b + 1], (length + back)[b:b + 1].contiguous(), None, 0, D ** -0.5, window, sinks)
        w, tol = want[b]
        assert ((got["out"][0].double() - w[prompts[b] - 1]).abs() <= tol[prompts[b] - 1]).all()
    # verify blocks behind them
    drafts = i32(np.arange(B + 1) * N)
    for step in range(steps):
        at = [p + step * (N + 1) for p in prompts]
        x = torch.cat([life[b][at[b]:at[b] + N + 1] for b in range(B)])
        a = sv.spec_cache_append_rotated(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pool[0][0], pool[1][0], table, length, t, cu_drafts=drafts, kmax=N)
        o = sv.spec_paged_attention(a["q"], pool[0][0], pool[1][0], table, length, drafts, N, D ** -0.5, window, sinks)
        assert (a["status"] == 0).all() and (o["status"] == 0).all()
        for b in range(B):
            w, tol = want[b]
            s = slice(at[b], at[b] + N + 1)
            assert ((o["out"][b * (N + 1):(b + 1) * (N + 1)].double() - w[s]).abs() <= tol[s]).all(), (step, b)
        sv.spec_cache_resize(*pool, *book, advance=i32([N + 1] * B), room=i32([N + 1] * B))
