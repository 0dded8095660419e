"""Calls on a stream that is not the current one: the buffers they make for themselves are that stream's."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


def attention():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    k, v = (torch.randn((260, 2, 16, 64), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, 8, 64), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.arange(260, dtype=torch.int32, device=DEV).view(2, 130)
    length = torch.tensor([2000, 1900], dtype=torch.int32, device=DEV)
    return lambda stream: sv.spec_paged_attention(q, k, v, table, length, None, 0, 0.125, stream=stream)


def append():
    k, v = torch.zeros((4, 1, 8, 8), device=DEV), torch.zeros((4, 1, 8, 8), device=DEV)
    new = torch.arange(16, dtype=torch.float32, device=DEV).view(2, 1, 8)
    table, length = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2), i32(2)
    return lambda stream: dict(sv.spec_cache_append(new, new, k, v, table, length, None, 0, stream=stream), k=k)


def resize():
    k, v = torch.zeros((1, 6, 1, 8, 8), device=DEV), torch.zeros((1, 6, 1, 8, 8), device=DEV)
    book = (i32(2, 3) - 1, i32(2), i32(2), i32(6))
    room = torch.tensor([9, 17], dtype=torch.int32, device=DEV)
    return lambda stream: dict(sv.spec_cache_resize(k, v, *book, room=room, stream=stream), table=book[0], refs=book[3])


def fork():
    book = (i32(2, 3) - 1, i32(2), i32(2), i32(6))
    src, dst = i32(1), i32(1) + 1
    return lambda stream: sv.spec_cache_fork(src, dst, *book, 8, stream=stream)


CALLS = [attention, append, resize, fork]


@pytest.mark.parametrize("make", CALLS, ids=lambda m: m.__name__)
def test_buffers_are_made_on_the_calls_stream(make, monkeypatch):
    call = make()
    side, made = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for name in ("empty", "zeros"):
        def record(*a, real=getattr(torch, name), **kw):
            made.append(torch.cuda.current_stream())
            return real(*a, **kw)
        monkeypatch.setattr(torch, name, record)
    before = torch.cuda.current_stream()
    call(side)
    side.synchronize()
    assert made and all(s == side for s in made)
    assert torch.cuda.current_stream() == before
    made.clear()
    call(None)
    assert made and all(s == before for s in made)


@pytest.mark.parametrize("make", CALLS, ids=lambda m: m.__name__)
def test_a_busy_current_stream_does_not_matter(make):
    want = {n: t.clone() for n, t in make()(None).items() if n != "workspace"}
    call = make()
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, device=DEV)
    # memory that the current stream has used and left full of ones
    for size in (1 << 9, 1 << 12, 1 << 16, 1 << 18, 1 << 20):
        left = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        del left
    torch.cuda.synchronize()
    for _ in range(60):
        busy.add_(1.0)
    got = call(side)
    side.synchronize()
    got = {n: t.cpu() for n, t in got.items() if n != "workspace"}
    for n, t in want.items():
        assert torch.equal(got[n], t.cpu()), n
