"""The cache calls at the ends of the sizes that they accept."""

import threading

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from tests import cache_reference as ref

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


def test_batches_of_different_sizes_from_several_threads():
    # above 12,288 streams the kernel needs its limit of shared memory raised, which is one for all threads
    failed = []

    def work(B):
        k = torch.zeros((1, 64, 1, 8, 8), dtype=torch.bfloat16, device=DEV)
        args = (k, k.clone(), i32(B, 1) - 1, i32(B), i32(B), i32(64))
        room = i32(B)
        out = sv.spec_cache_resize(*args, room=room)
        for _ in range(2000):
            try:
                sv.spec_cache_resize(*args, room=room, out=out)
            except sv.SpecError as e:
                failed.append((B, str(e)))

    threads = [threading.Thread(target=work, args=(B,)) for B in (16000, 65000, 30000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])


@pytest.mark.parametrize("B,width", [(12289, 3), (20001, 2), (65535, 1)])
def test_resize_of_many_streams(B, width):
    # against the page-by-page model; several streams a thread, and shared memory above the default limit
    P, rng = 8, np.random.default_rng(B)
    pages = int(1.2 * B)
    k = torch.arange(pages, dtype=torch.float32, device=DEV).view(1, pages, 1, 1, 1).expand(1, pages, 1, P, 8).contiguous()
    v = -k
    book = (i32(B, width) - 1, i32(B), i32(B), i32(pages))
    model = ref.Book(book[0].tolist(), [0] * B, [0] * B, [0] * pages, P, range(pages))

    def same(advance, room):
        d = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        got = sv.spec_cache_resize(k, v, *book, advance=d(advance), room=d(room))["status"].tolist()
        assert got == model.resize(advance, room)
        for t, m in zip(book, (model.table, model.held, model.length, model.refs)):
            assert t.tolist() == m
        contents = torch.tensor(model.contents, dtype=torch.float32, device=DEV)
        assert torch.equal(k[0, :, 0, 0, 0], contents) and torch.equal(v, -k)

    same(None, (rng.random(B) < 0.5).astype(int).tolist())
    same([int(h > 0) for h in model.held], None)
    src = [b for b in range(B) if model.length[b]][:300]
    dst = [b for b in range(B) if not model.length[b]][-300:]
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    assert sv.spec_cache_fork(d(src), d(dst), *book, P)["status"].tolist() == model.fork(src, dst)
    same(None, rng.integers(0, (width - 1) * P + 4, B).tolist())
    same([-n for n in model.length], [1] * B)
