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


def verify_inputs():
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    q, p = (torch.randn((n, 512), generator=g, device=DEV) for n in (5, 7))
    x = torch.randint(0, 512, (5,), generator=g, device=DEV, dtype=torch.int32)
    return cu, q, p, x, torch.ones(2, device=DEV)


def verify(call, **kw):
    def make():
        cu, q, p, x, T = verify_inputs()
        return lambda stream: call(cu, q, p, x, T, 3, 11, 0, diag=True, stream=stream, **kw)
    make.__name__ = call.__name__
    return make


def verify_reduced():
    cu, q, p, x, T = verify_inputs()
    t2d = torch.arange(512, dtype=torch.int32, device=DEV)
    return lambda stream: sv.spec_verify_block_reduced(cu, q, t2d, p, x, T, 3, 11, 0, stream=stream)


def markov():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    base, W1, W2 = (torch.randn(s, generator=g, device=DEV) for s in ((2, 3, 512), (512, 16), (16, 512)))
    return base, torch.tensor([5, 9], dtype=torch.int32, device=DEV), W1, W2, torch.ones(2, device=DEV)


def walk():
    base, anchor, W1, W2, T = markov()
    return lambda stream: sv.dspark_markov_walk(base, anchor, W1, W2, T, 4, 0, stream=stream)


def bias():
    base, anchor, W1, W2, _ = markov()
    rows = base[:, 0].contiguous()
    return lambda stream: {"out": sv.dspark_markov_bias(rows, anchor, W1, W2, stream=stream)}


def pick():
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    hidden, w = torch.randn((3, 4, 64), generator=g, device=DEV), torch.randn(64, generator=g, device=DEV)
    ms = torch.linspace(1.0, 2.0, 32, device=DEV)
    return lambda stream: sv.adaptive_pick_k(hidden, w, 0.1, ms, stream=stream)


def counters():
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    accepted = torch.tensor([2, 1], dtype=torch.int32, device=DEV)
    status = i32(2)
    return lambda stream: {"counts": sv.spec_accept_counters(accepted, status, cu, 3, stream=stream)}


def philox():
    return lambda stream: {"out": sv.spec_philox_uniforms(1, 2, 3, 4, stream=stream)}


CALLS = [attention, append, resize, fork, verify(sv.spec_verify_block), verify(sv.spec_verify_tokenwise),
         verify(sv.spec_verify_block_static), verify_reduced, walk, bias, pick, counters, philox]


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
    want = {n: t.float() if t.dtype == torch.bfloat16 else t.clone() for n, t in make()(None).items() if n != "workspace"}
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
    got = {n: t.float().cpu() if t.dtype == torch.bfloat16 else t.cpu() for n, t in got.items() if n != "workspace"}
    for n, t in want.items():
        assert got[n].numpy().tobytes() == t.cpu().numpy().tobytes(), n   # bit for bit, NaN too
