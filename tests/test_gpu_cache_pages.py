"""spec_cache_resize and spec_cache_fork against a page-by-page model: every integer equal, and the
contents of copied pages bit for bit."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


class Pair:
    """The device's cache and the model's, kept side by side."""

    def __init__(self, B, width, pages, P=8, layers=2, Hkv=1, D=8, dtype=torch.bfloat16):
        self.P = P
        self.k = torch.arange(layers * pages, device=DEV).view(layers, pages, 1, 1, 1).to(torch.float32)
        self.k = (self.k + 0.5 * torch.arange(Hkv * P * D, device=DEV).view(1, 1, Hkv, P, D) / (Hkv * P * D)).to(dtype).contiguous()
        self.v = -self.k
        self.k0, self.v0 = self.k.clone(), self.v.clone()
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
        self.table, self.held, self.length, self.refs = i32(B, width) - 1, i32(B), i32(B), i32(pages)
        self.book = self.model()

    def model(self):
        return ref.Book(self.table.tolist(), self.held.tolist(), self.length.tolist(), self.refs.tolist(), self.P,
                        range(self.refs.numel()))

    def args(self):
        return self.table, self.held, self.length, self.refs

    def resize(self, advance=None, room=None):
        d = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        got = sv.spec_cache_resize(self.k, self.v, *self.args(), advance=d(advance), room=d(room))["status"].tolist()
        want = self.book.resize(advance, room)
        assert got == want, (got, want)
        self.same()
        return got

    def fork(self, src, dst):
        d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        got = sv.spec_cache_fork(d(src), d(dst), *self.args(), self.P)["status"].tolist()
        want = self.book.fork(src, dst)
        assert got == want, (got, want)
        self.same()
        return got

    def same(self):
        m = self.book
        assert self.table.tolist() == m.table
        assert self.held.tolist() == m.held and self.length.tolist() == m.length and self.refs.tolist() == m.refs
        src = torch.tensor(m.contents, device=DEV)
        assert torch.equal(self.k, self.k0[:, src]) and torch.equal(self.v, self.v0[:, src])

    def consistent(self):
        """Every count is the number of holders."""
        n = np.zeros(self.refs.numel(), np.int64)
        for row, h in zip(self.table.tolist(), self.held.tolist()):
            for p in row[:h]:
                n[p] += 1
            assert all(p == -1 for p in row[h:])
        assert n.tolist() == self.refs.tolist()


def test_reserve_commit_release():
    c = Pair(5, 12, 40)
    c.resize(room=[0, 1, 8, 9, 30])
    assert c.held.tolist() == [0, 1, 1, 2, 4]
    c.resize(advance=[0, 1, 3, 9, 17])
    assert c.held.tolist() == [0, 1, 1, 2, 3]
    c.resize(advance=[0, 0, 5, -4, 0], room=[6] * 5)
    c.resize(advance=[0, -1, -8, -5, -17])
    assert c.refs.sum() == 0 and (c.table == -1).all()


@pytest.mark.parametrize("B,pages,P,width", [(1, 9, 8, 8), (3, 20, 16, 6), (64, 700, 8, 12), (700, 5000, 8, 9), (5000, 9000, 8, 4)])
def test_random_walks(B, pages, P, width):
    rng = np.random.default_rng(B)
    c = Pair(B, width, pages, P=P, layers=1)
    for _ in range(8 if B < 1000 else 4):
        room = rng.integers(0, 3 * P, B)
        c.resize(room=room.tolist())
        # what fits is kept: up to the held pages, some of it rolled back
        top = c.held.cpu().numpy() * P - c.length.cpu().numpy()
        advance = np.minimum(rng.integers(0, 2 * P, B), top)
        back = rng.random(B) < 0.2
        advance[back] = -rng.integers(0, c.length.cpu().numpy()[back] + 1)
        if rng.random() < 0.5:
            c.resize(advance=advance.tolist())
        else:
            c.resize(advance=advance.tolist(), room=rng.integers(0, P, B).tolist())
        c.consistent()
        if B > 2:
            m = int(rng.integers(1, max(2, B // 2)))
            who = rng.permutation(B)
            src, dst = who[:m // 2 + 1], who[m // 2 + 1:m + 1]
            if len(dst):
                c.fork(rng.choice(src, len(dst)).tolist(), dst.tolist())
                c.consistent()


@pytest.mark.parametrize("length", [1, 8, 13, 16])
@pytest.mark.parametrize("children", [1, 4])
def test_fork_and_copy_on_write(length, children):
    c = Pair(1 + children, 8, 64, Hkv=2, D=16)
    c.resize(room=[length + 3] + [0] * children)
    c.resize(advance=[length] + [0] * children, room=[3] + [0] * children)
    c.fork([0] * children, list(range(1, children + 1)))
    assert c.refs.max() == 1 + children
    c.resize()                                   # no room: nothing is copied
    assert torch.equal(c.k, c.k0)
    c.resize(room=[0] + [6] * children)          # the parent keeps the page, every child gets a copy
    c.consistent()
    c.resize(advance=[0] + [6] * children)
    c.fork([0] * children, list(range(1, children + 1)))   # a child is replaced
    c.resize(room=[2] * (1 + children))          # all of them ask: the lowest keeps the page
    c.consistent()


def test_fork_then_roll_back_into_shared_pages():
    c = Pair(4, 10, 60)
    c.resize(room=[50, 0, 0, 0])
    c.resize(advance=[50, 0, 0, 0])
    c.fork([0, 0], [1, 2])
    c.resize(advance=[0, -27, -27, 0], room=[0, 9, 20, 5])   # positions past 23 are written anew
    c.consistent()
    c.resize(advance=[-50, 0, 0, 0])
    c.resize(advance=[0, -23, -23, 0])
    assert c.refs.tolist().count(0) == 60


def test_too_few_pages():
    c = Pair(4, 10, 10)
    assert c.resize(room=[30, 30, 10, 8]) == [0, 0, 0, 8]
    c.resize(advance=[30, 3, 1, 0])
    c.fork([0], [3])
    assert c.resize(room=[1, 60, 1, 1]) == [0, 8, 0, 8]
    c.consistent()
    assert c.resize(advance=[0, -3, 0, 0], room=[0, 0, 0, 1])[3] == 0
    c.consistent()


def test_statuses_leave_streams_alone():
    c = Pair(6, 4, 30)
    c.resize(room=[10] * 6)
    assert c.resize(advance=[17, -1, 0, 0, 3, 0], room=[0, 0, -1, 33, 5, 32]) == [9, 9, 9, 9, 0, 0]
    c.table[1, 1] = 30
    c.book.table[1][1] = 30
    c.held[2] = 5
    c.book.held[2] = 5
    assert c.resize(room=[1, 1, 1, 1, 1, 1])[1:3] == [10, 9]
    assert c.fork([0, 0, 1, 0, 6, 0, 4], [3, 3, 5, 2, 0, -1, 4]) == [0, 11, 0, 9, 11, 11, 11]
    c.table[1, 0] = -7
    c.book.table[1][0] = -7
    c.resize(advance=[0, 3, 0, 0, 0, 0], room=[0, 9, 0, 0, 0, 0])


def test_long_tables_and_unaligned_counts():
    c = Pair(3, 3000, 9001, layers=1)
    flat = torch.zeros(9002, dtype=torch.int32, device=DEV)
    c.refs = flat[1:]
    c.resize(room=[23000, 17, 23999])
    c.resize(advance=[20001, 17, 23999])
    c.fork([0], [1])
    c.resize(advance=[-20001, 0, -23999])
    c.resize(room=[1, 1, 1])
    c.consistent()


def test_pool_of_many_scans():
    # the free pages lie beyond the first pass over the counts
    c = Pair(2, 64, 200000, layers=1)
    c.refs[:199990] = 1
    c.book = c.model()
    assert c.resize(room=[20, 70]) == [0, 8]
    assert c.table[0, :3].tolist() == [199990, 199991, 199992]


def test_graph_of_a_step():
    c = Pair(3, 20, 60)
    room = torch.tensor([6, 6, 6], dtype=torch.int32, device=DEV)
    kept = torch.tensor([1, 6, 3], dtype=torch.int32, device=DEV)
    a = sv.spec_cache_resize(c.k, c.v, *c.args(), room=room)
    b = sv.spec_cache_resize(c.k, c.v, *c.args(), advance=kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_cache_resize(c.k, c.v, *c.args(), room=room, out=a)
        sv.spec_cache_resize(c.k, c.v, *c.args(), advance=kept, out=b)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for _ in range(6):
        assert c.book.resize(room=[6, 6, 6]) == [0, 0, 0]
        c.book.resize(advance=[1, 6, 3])
    c.same()


def test_refusals():
    c = Pair(2, 4, 10)
    with pytest.raises(TypeError):
        sv.spec_cache_resize(c.k, c.v, c.table.long(), c.held, c.length, c.refs)
    with pytest.raises(ValueError):
        sv.spec_cache_resize(c.k[:, :5], c.v[:, :5], *c.args())
    with pytest.raises(ValueError):
        sv.spec_cache_resize(c.k, c.v, *c.args(), room=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        sv.spec_cache_resize(c.k, c.v, c.table, c.held[:1], c.length, c.refs)
    out = sv.spec_cache_resize(c.k, c.v, *c.args())
    with pytest.raises(sv.SpecError) as e:
        sv.spec_cache_resize(c.k, c.v, *c.args(), out=dict(out, workspace=out["workspace"][:64]))
    assert e.value.code == -6
    odd = torch.zeros((1, 10, 1, 12, 8), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_cache_resize(odd, odd, *c.args())
    with pytest.raises(sv.SpecError):
        sv.spec_cache_fork(c.held[:1], c.held[:1], *c.args(), 12)
    with pytest.raises(TypeError):
        sv.spec_cache_fork(c.held[:1].long(), c.held[:1], *c.args(), 8)
    with pytest.raises(TypeError):
        sv.spec_cache_fork(c.held[:1].cpu(), c.held[:1], *c.args(), 8)
    assert sv.spec_cache_fork(c.held[:0], c.held[:0], *c.args(), 8)["status"].numel() == 0
