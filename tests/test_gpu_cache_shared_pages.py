"""A page that several streams hold is not written into by a stream that resize had no page for, in a loop that hands
resize's statuses to append and reads neither."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def d(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def forked(pages, P=8, tokens=13, Hkv=2, D=8, dtype=torch.float32):
    """Stream 0 with 13 tokens (two pages), streams 1 and 2 its continuations."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    c = dict(k=torch.randn((1, pages, Hkv, P, D), device=DEV).to(dtype), table=i32(3, 4) - 1, held=i32(3), length=i32(3), refs=i32(pages))
    c["v"] = -c["k"]
    c["book"] = book = (c["table"], c["held"], c["length"], c["refs"])
    assert sv.spec_cache_resize(c["k"], c["v"], *book, room=d(tokens, 0, 0))["status"].tolist() == [0, 0, 0]
    assert sv.spec_cache_resize(c["k"], c["v"], *book, advance=d(tokens, 0, 0))["status"].tolist() == [0, 0, 0]
    assert sv.spec_cache_fork(d(0, 0), d(1, 2), *book, P)["status"].tolist() == [0, 0]
    return c


def append(c, new, cu, reserved):
    return sv.spec_cache_append(new, -new, c["k"][0], c["v"][0], c["table"], c["length"], cu, 1, reserved=reserved)["status"].tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [0, 1])
def test_a_stream_without_its_copy_leaves_the_shared_page_alone(extra, dtype):
    # one free page: stream 1 gets its copy, stream 2 does not and still shares its second page with stream 0
    c = forked(3, dtype=dtype)
    r = sv.spec_cache_resize(c["k"], c["v"], *c["book"], room=d(2, 2, 2))["status"]
    assert r.tolist() == [0, 0, 8]
    page = [int(c["table"][b, 1]) for b in range(3)]
    assert page[0] == page[2] != page[1] and c["refs"].tolist()[page[0]] == 2
    cu = d(0, 1, 2, 3)   # two tokens each
    wide = torch.randn(6 * 16 + 1, device=DEV).to(dtype)
    new = wide[extra:extra + 96].view(6, 2, 8)   # extra 1: the element-wise form
    k, v = c["k"].clone(), c["v"].clone()
    assert append(c, new, cu, r) == [0, 0, 8]
    for b in (0, 1):
        for i in range(2):
            k[0, page[b], :, (13 + i) % 8] = new[2 * b + i]
            v[0, page[b], :, (13 + i) % 8] = -new[2 * b + i]
    assert torch.equal(c["k"], k) and torch.equal(c["v"], v)
    # stream 1 ends: now there is a page for stream 2, which begins with its own five tokens
    r = sv.spec_cache_resize(c["k"], c["v"], *c["book"], advance=d(2, -13, 0), room=d(0, 0, 2))["status"]
    assert r.tolist() == [0, 0, 0]
    mine = int(c["table"][2, 1])
    assert mine != page[0] and c["refs"].tolist()[page[0]] == 1
    assert torch.equal(c["k"][0, mine, :, :5], k[0, page[0], :, :5])
    assert append(c, new, cu, d(0, 9, 0)) == [10, 9, 0]   # stream 0 has no room left, stream 1 is passed over
    assert torch.equal(c["k"][0, page[0], :, :7], k[0, page[0], :, :7])
    assert torch.equal(c["k"][0, mine, :, 5:7], new[4:6].transpose(0, 1))


@pytest.mark.parametrize("back,status", [(0, 0), (1, 8), (4, 8)])
def test_the_holder_that_may_write_does_not_overwrite_longer_ones(back, status):
    # no free page; stream 0 is rolled back by `back` tokens and keeps the page that the others, all of them asking
    # for a copy, still have up to 13 tokens in
    c = forked(2)
    r = sv.spec_cache_resize(c["k"], c["v"], *c["book"], advance=d(-back, 0, 0), room=d(2, 2, 2))["status"]
    assert r.tolist() == [0, 8, 8]
    new = torch.randn((6, 2, 8), device=DEV)
    k, page = c["k"].clone(), int(c["table"][0, 1])
    assert append(c, new, d(0, 1, 2, 3), r) == [status, 8, 8]
    if status == 0:
        k[0, page, :, 5:7] = new[:2].transpose(0, 1)
    assert torch.equal(c["k"], k)


def test_many_streams_beside_the_one_that_waits():
    # the sibling is stream 699 of 700: looked for by every thread of the block
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    B, P = 700, 8
    k = torch.randn((1, 2, 1, P, 8), device=DEV)
    v = k.clone()
    book = (table, held, length, refs) = (i32(B, 2) - 1, i32(B), i32(B), i32(2))
    first, none = i32(B), i32(B)
    first[0] = 5
    sv.spec_cache_resize(k, v, *book, room=first)
    sv.spec_cache_resize(k, v, *book, advance=first)
    sv.spec_cache_fork(d(0), d(B - 1), *book, P)
    refs[1] = 1   # somebody else's
    none[0] = -2
    room = i32(B)
    room[0] = room[B - 1] = 2
    r = sv.spec_cache_resize(k, v, *book, advance=none, room=room)["status"]
    assert r.tolist() == [0] * (B - 1) + [8]
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    new = torch.randn((2 * B, 1, 8), device=DEV)
    before = k.clone()
    got = sv.spec_cache_append(new, new, k[0], v[0], table, length, cu, 1, reserved=r)["status"].tolist()
    assert got == [8] + [10] * (B - 2) + [8] and torch.equal(k, before)


def test_broken_offsets_come_first():
    c = forked(3)
    new = torch.randn((6, 2, 8), device=DEV)
    k = c["k"].clone()
    assert append(c, new, d(1, 1, 2, 3), d(0, 8, 8)) == [5, 5, 5]
    assert append(c, new, d(0, 1, 2, 3), d(8, 9, 10)) == [8, 9, 10]
    assert torch.equal(c["k"], k)


def test_refusals():
    c = forked(3)
    new = torch.randn((6, 2, 8), device=DEV)
    r = d(0, 0, 0)
    with pytest.raises(ValueError):
        append(c, new, d(0, 1, 2, 3), r[:2])
    with pytest.raises(TypeError):
        append(c, new, d(0, 1, 2, 3), r.long())
    with pytest.raises(TypeError):
        append(c, new, d(0, 1, 2, 3), r.cpu())
