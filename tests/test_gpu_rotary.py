"""spec_rotate and spec_cache_append_rotated against the definitions in 64 bits (tolerances: prompt_reference)."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import prompt_reference as ref  # noqa: E402

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
MARK = -77.0


def rand(seed, shape, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def close(got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (float((off / tol.clamp(min=1e-300)).max()), bad.nonzero()[:4].tolist(), int(bad.sum()))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,dim", [(64, 64), (128, 128), (128, 64), (80, 20), (80, 80), (8, 2), (8, 8), (96, 42), (256, 256), (256, 250), (72, 16), (136, 6)])
def test_heads_and_parts(D, dim, inter, dtype):
    x = rand(1, (37, 5, D), dtype)
    at = i32(np.random.default_rng(2).integers(0, 5000, 37).tolist())
    t = sv.RotaryTable(dim, interleaved=inter)
    want, tol = ref.rotate(x, at, ref.frequencies(dim), 1.0, inter)
    got = sv.spec_rotate(x, at, t)
    close(got, want, tol)
    assert torch.equal(got[..., dim:], x[..., dim:])
    # slices of a wider projection, in and out, and in place
    wide = rand(3, (37, 9, D), dtype)
    wide[:, 2:7] = x
    into = torch.full((37, 8, D), MARK, dtype=dtype, device=DEV)
    sv.spec_rotate(wide[:, 2:7], at, t, out=into[:, 1:6])
    assert torch.equal(into[:, 1:6], got) and (into[:, 0] == MARK).all() and (into[:, 6:] == MARK).all()
    rest = wide.clone()
    sv.spec_rotate(wide[:, 2:7], at, t, out=wide[:, 2:7])
    assert torch.equal(wide[:, 2:7], got) and torch.equal(wide[:, :2], rest[:, :2]) and torch.equal(wide[:, 7:], rest[:, 7:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scaling,base,factor,original", [("none", 1e4, 1.0, 4096), ("linear", 1e4, 4.0, 4096), ("ntk", 1e4, 8.0, 4096), ("yarn", 5e5, 16.0, 8192),
                                                          ("yarn", 1e4, 1.0, 2048)])
def test_scalings_at_far_positions(scaling, base, factor, original, dtype):
    x = rand(4, (64, 3, 128), dtype)
    at = i32([0, 1, 2, 3, 131071, 131072, 1000003, 16777217, 2147483647, -1, -5, -1000003] + list(range(100, 100 * 53, 100)))
    t = sv.RotaryTable(128, base=base, scaling=scaling, factor=factor, original=original)
    m = 0.1 * np.log(factor) + 1 if scaling == "yarn" else 1.0
    want, tol = ref.rotate(x, at, ref.frequencies(128, base, scaling, factor, original), m)
    close(sv.spec_rotate(x, at, t), want, tol)


def test_turning_back():
    x = rand(5, (50, 4, 64), F32)
    at = i32(list(range(0, 50 * 997, 997)))
    t = sv.RotaryTable(64)
    back = sv.spec_rotate(sv.spec_rotate(x, at, t), -at, t)
    norm = (x[..., :32].abs() + x[..., 32:].abs()).repeat(1, 1, 2)
    assert ((back - x).abs() <= 2 * 2 * 10 * 2.0 ** -24 * norm).all()   # two turns, each off by 10 u of |a| + |b| and mixed once more


@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 72), (6, 20), (7, 4096), (300, 1), (2049, 72), (8191, 9)])
@pytest.mark.parametrize("inter", [False, True])
def test_sizes(rows, heads, inter):
    x = rand(6, (rows, heads, 64), BF16)
    at = i32(np.random.default_rng(7).integers(0, 100000, rows).tolist())
    want, tol = ref.rotate(x, at, ref.frequencies(64), 1.0, inter)
    close(sv.spec_rotate(x, at, sv.RotaryTable(64, interleaved=inter)), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rows_off_16_byte_boundaries(inter, dtype):
    flat = rand(8, (11 * 321 + 5,), dtype)
    x = torch.as_strided(flat, (11, 5, 64), (321, 64, 1), 3)
    at = i32(list(range(11)))
    want, tol = ref.rotate(x, at, ref.frequencies(64), 1.0, inter)
    close(sv.spec_rotate(x, at, sv.RotaryTable(64, interleaved=inter)), want, tol)


def test_given_frequencies_and_what_is_not_finite():
    x = rand(9, (4, 2, 8), F32)
    x[1, 0, 0], x[2, 1, 7] = float("nan"), float("inf")
    t = sv.RotaryTable(4, frequencies=[0.3, 7.5], magnitude=0.5)
    got = sv.spec_rotate(x, i32([3, 4, 5, 6]), t)
    want, tol = ref.rotate(x, i32([3, 4, 5, 6]), [0.3, 7.5], 0.5)
    fine = torch.isfinite(want)
    close(got[fine], want[fine], tol[fine])
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and got[2, 1, 7] == float("inf")


def test_empty_and_refused():
    t = sv.RotaryTable(64)
    assert sv.spec_rotate(torch.empty((0, 3, 64), device=DEV), i32([]), t).shape == (0, 3, 64)
    x = rand(10, (4, 3, 64), F32)
    at = i32([0, 1, 2, 3])
    for args, what in [((x.cpu(), at, t), TypeError), ((x.half(), at, t), TypeError), ((x[0], at, t), ValueError), ((x, at[:3], t), ValueError), ((x, at.long(), t), TypeError),
                       ((x.transpose(0, 1), at, t), ValueError), ((x[..., :32], at, t), ValueError), ((x[..., :32].contiguous(), at, t), sv.SpecError),
                       ((x, at, sv.RotaryTable(64, device="cpu")), ValueError)]:
        with pytest.raises(what):
            sv.spec_rotate(*args)
    with pytest.raises(ValueError):
        sv.spec_rotate(x, at, t, out=torch.empty((3, 3, 64), device=DEV))


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
def make(seed, length, rows, Hq, Hkv, D, P, dtype, behind=2, spare=3, table=None):
    rng = np.random.default_rng(seed)
    B, n = len(rows), sum(rows)
    need = [-(-(max(a, 0) + r) // P) for a, r in zip(length, rows)]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    t = np.full((B, max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        t[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    wide = rand(seed, (n + behind, Hq + 2 * Hkv, D), dtype)
    pool = lambda: torch.full((pages, Hkv, P, D), MARK, dtype=dtype, device=DEV)  # noqa: E731
    return dict(q=wide[:, :Hq], k=wide[:, Hq:Hq + Hkv], v=wide[:, Hq + Hkv:], kp=pool(), vp=pool(), table=i32(t.tolist()), t=t,
                length=i32(list(length)), len=list(length), rows=list(rows), cu=[0] + list(np.cumsum(rows)), P=P)


def outs(c, keep=True):
    like = lambda x: torch.full(x.shape, MARK, dtype=x.dtype, device=DEV)  # noqa: E731
    return {"q": like(c["q"]), "k": like(c["k"]) if keep else None, "status": torch.full((len(c["rows"]),), 99, dtype=torch.int32, device=DEV)}


def check(c, got, f, m=1.0, inter=False, skip=(), keep=True, skip_pages=()):
    """Everything is where it belongs, and all else as it was."""
    n, P = c["cu"][-1], c["P"]
    at = torch.tensor(ref.positions_of(c["cu"], c["len"]), device=DEV)
    q, qt = ref.rotate(c["q"][:n], at, f, m, inter)
    k, kt = ref.rotate(c["k"][:n], at, f, m, inter)
    kp, vp = torch.full(c["kp"].shape, MARK, dtype=torch.float64, device=DEV), torch.full(c["vp"].shape, MARK, dtype=torch.float64, device=DEV)
    kpt = torch.zeros_like(kp)
    there = torch.zeros(c["q"].shape[0], dtype=torch.bool, device=DEV)
    r = 0
    for b, rows in enumerate(c["rows"]):
        for i in range(rows):
            p = c["len"][b] + i
            if b not in skip:
                there[r] = True
                page = c["t"][b, p // P]
                if page not in skip_pages:
                    kp[page, :, p % P], kpt[page, :, p % P], vp[page, :, p % P] = k[r], kt[r], c["v"][r].double()
            r += 1
    close(c["kp"], kp, kpt)
    assert torch.equal(c["vp"].double(), vp)
    close(got["q"][:n][there[:n]], q[there[:n]], qt[there[:n]])
    assert (got["q"][~there] == MARK).all()
    if keep:
        close(got["k"][:n][there[:n]], k[there[:n]], kt[there[:n]])
        assert (got["k"][~there] == MARK).all()


def call(c, t, **kw):
    if "cu_rows" not in kw:
        kw["cu_rows"] = i32(c["cu"])
    return sv.spec_cache_append_rotated(c["q"], c["k"], c["v"], c["kp"], c["vp"], c["table"], c["length"], t, **kw)


CASES = [(64, 64, False), (128, 128, False), (128, 64, True), (80, 20, False), (80, 32, True), (8, 2, False), (256, 256, False), (256, 254, True), (96, 48, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,dim,inter", CASES)
def test_append_heads(D, dim, inter, dtype):
    c = make(11, [0, 5, 130, 16, 47, 0], [40, 0, 7, 1, 3, 129], 6, 2, D, 16, dtype)
    t = sv.RotaryTable(dim, scaling="yarn", factor=4.0, original=64, interleaved=inter)
    got = call(c, t, out=outs(c), keep_keys=True)
    assert got["status"].tolist() == [0] * 6
    check(c, got, ref.frequencies(dim, scaling="yarn", factor=4.0, original=64), 0.1 * np.log(4.0) + 1, inter)


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("keep", [False, True])
def test_append_pages(P, keep):
    lengths = [0, 1, P - 1, P, P + 1, 3 * P - 2, 1000]
    c = make(12, lengths, [1, P, P + 1, 2, 0, 5, 3 * P], 4, 1, 64, P, BF16)
    got = call(c, sv.RotaryTable(64), out=outs(c, keep), keep_keys=keep)
    assert (got["status"] == 0).all()
    check(c, got, ref.frequencies(64), keep=keep)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_long_prompts(dtype):
    c = make(13, [0, 17, 0], [2500, 1, 1333], 16, 4, 128, 16, dtype)
    got = call(c, sv.RotaryTable(128), out=outs(c), keep_keys=True)
    check(c, got, ref.frequencies(128))


@pytest.mark.parametrize("kmax", [0, 5, 100])
@pytest.mark.parametrize("given", [False, True])
def test_append_blocks(kmax, given):
    drafts = [kmax, 0, kmax // 2, kmax] if given else [kmax] * 4
    c = make(14, [3, 100, 0, 15], [d + 1 for d in drafts], 8, 2, 64, 16, BF16, behind=2 if given else 0)
    got = call(c, sv.RotaryTable(64), cu_rows=None, cu_drafts=i32([0] + list(np.cumsum(drafts))) if given else None, kmax=kmax, out=outs(c), keep_keys=True)
    assert (got["status"] == 0).all()
    check(c, got, ref.frequencies(64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_append_equals_rotate_and_append(inter, dtype):
    a = make(15, [7, 64, 0], [6, 1, 4], 8, 2, 128, 16, dtype, behind=0)
    b = make(15, [7, 64, 0], [6, 1, 4], 8, 2, 128, 16, dtype, behind=0)
    t = sv.RotaryTable(128, interleaved=inter)
    got = call(a, t, keep_keys=True)
    at = i32(ref.positions_of(b["cu"], b["len"]))
    k = sv.spec_rotate(b["k"], at, t)
    sv.spec_cache_append(k, b["v"], b["kp"], b["vp"], b["table"], b["length"], i32([0, 5, 5, 8]), 5)
    assert torch.equal(a["kp"], b["kp"]) and torch.equal(a["vp"], b["vp"]) and torch.equal(got["k"], k)
    assert torch.equal(got["q"], sv.spec_rotate(b["q"], at, t))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_append_off_16_byte_boundaries(inter, dtype):
    c = make(16, [3, 0], [6, 20], 4, 2, 64, 16, dtype, behind=0)
    flat = rand(17, (26 * 515 + 9,), dtype)
    for name, heads, first in (("q", 4, 1), ("k", 2, 257), ("v", 2, 386)):
        c[name] = torch.as_strided(flat, (26, heads, 64), (515, 64, 1), first)
    got = call(c, sv.RotaryTable(64, interleaved=inter), out=outs(c), keep_keys=True)
    check(c, got, ref.frequencies(64), 1.0, inter)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_in_place_and_without_queries(dtype):
    c = make(18, [5, 0], [9, 30], 4, 2, 64, 8, dtype)
    d = make(18, [5, 0], [9, 30], 4, 2, 64, 8, dtype)
    t = sv.RotaryTable(64)
    want = call(c, t, keep_keys=True)
    n = c["cu"][-1]
    got = call(d, t, keep_keys=True, out={"q": d["q"], "k": d["k"], "status": torch.zeros(2, dtype=torch.int32, device=DEV)})
    assert torch.equal(got["q"][:n], want["q"][:n]) and torch.equal(d["k"][:n], want["k"][:n]) and torch.equal(c["kp"], d["kp"])
    assert torch.equal(d["q"][n:], c["q"][n:])
    e = make(18, [5, 0], [9, 30], 4, 2, 64, 8, dtype)
    out = sv.spec_cache_append_rotated(None, e["k"], e["v"], e["kp"], e["vp"], e["table"], e["length"], t, cu_rows=i32(e["cu"]))
    assert out["q"] is None and out["k"] is None and torch.equal(e["kp"], c["kp"]) and torch.equal(e["vp"], c["vp"])


def test_append_many_streams():
    rng = np.random.default_rng(19)
    for B in (255, 300, 2000):
        c = make(20, rng.integers(0, 50, B).tolist(), rng.integers(0, 7, B).tolist(), 2, 1, 64, 8, BF16)
        got = call(c, sv.RotaryTable(64), out=outs(c), keep_keys=True)
        assert (got["status"] == 0).all()
        check(c, got, ref.frequencies(64))


def test_append_statuses():
    # 1: length negative; 3: past its table row; 5: a page that is not in the pool
    c = make(21, [4, 20, 0, 30, 9, 40], [3, 2, 20, 5, 1, 12], 4, 2, 64, 16, BF16)
    c["length"][1] = -1
    c["length"][3] = c["table"].shape[1] * 16 - 4
    bad = int(c["t"][5, 3])
    c["table"][5, 3] = 10 ** 6
    got = call(c, sv.RotaryTable(64), out=outs(c), keep_keys=True)
    assert got["status"].tolist() == [0, 9, 0, 9, 0, 10]
    check(c, got, ref.frequencies(64), skip=(1, 3), skip_pages=(bad,))


@pytest.mark.parametrize("cu,first", [([1, 3, 6], 0), ([0, 4, 3], 1), ([0, 3, 9], 1), ([0, 3, 6, 5, 8], 2), ([-1, 3, 5], 0)])
def test_append_broken_offsets(cu, first):
    B = len(cu) - 1
    rows = [max(0, cu[b + 1] - cu[b]) if b < first else 0 for b in range(B)]
    c = make(22, [5] * B, rows, 4, 2, 64, 16, BF16, behind=8 - sum(rows))   # 8 rows
    got = call(c, sv.RotaryTable(64), cu_rows=i32(cu), out=outs(c), keep_keys=True)
    assert got["status"].tolist() == [0 if b < first else 5 for b in range(B)]
    check(c, got, ref.frequencies(64))


def test_append_block_longer_than_kmax():
    c = make(23, [5, 5, 5], [3, 0, 0], 4, 2, 64, 16, BF16, behind=10)
    got = call(c, sv.RotaryTable(64), cu_rows=None, cu_drafts=i32([0, 2, 6, 7]), kmax=3, out=outs(c), keep_keys=True)
    assert got["status"].tolist() == [0, 5, 5]
    check(c, got, ref.frequencies(64))


def test_append_reserved():
    # stream 1 found no page; stream 2 shares its last page with stream 1, which keeps more tokens in it
    c = make(24, [5, 30, 20, 33], [3, 2, 4, 1], 4, 2, 64, 16, BF16)
    c["t"][2, 1] = c["t"][1, 1]
    c["table"][2, 1] = c["table"][1, 1]
    reserved = i32([0, 8, 0, 0])
    got = call(c, sv.RotaryTable(64), out=outs(c), keep_keys=True, reserved=reserved)
    assert got["status"].tolist() == [0, 8, 8, 0]
    check(c, got, ref.frequencies(64), skip=(1, 2))
    # the same from the plain append
    d = make(24, [5, 30, 20, 33], [3, 2, 4, 1], 4, 2, 64, 16, BF16, behind=0)
    d["table"][2, 1] = d["table"][1, 1]
    plain = sv.spec_cache_append(d["k"], d["v"], d["kp"], d["vp"], d["table"], d["length"], i32([0, 2, 3, 6, 6]), 3, reserved=reserved)
    assert torch.equal(plain["status"], got["status"])


def test_append_no_rows():
    c = make(25, [5, 30], [0, 0], 4, 2, 64, 16, BF16, behind=0)
    got = call(c, sv.RotaryTable(64), keep_keys=True)
    assert got["status"].tolist() == [0, 0] and got["q"].shape == (0, 4, 64)
    assert (c["kp"] == MARK).all()
    c["length"][1] = -3
    assert call(c, sv.RotaryTable(64))["status"].tolist() == [0, 9]


def test_append_on_another_stream_and_replayed():
    c = make(26, [5, 300, 0], [60, 6, 500], 8, 2, 128, 16, BF16)
    t = sv.RotaryTable(128)
    want = call(c, t, keep_keys=True)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    n = c["cu"][-1]
    cu = i32(c["cu"])
    side = torch.cuda.Stream()
    c["kp"].fill_(MARK)
    c["vp"].fill_(MARK)
    side.wait_stream(torch.cuda.current_stream())
    out = call(c, t, keep_keys=True, stream=side, cu_rows=cu)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c["kp"], kp) and torch.equal(c["vp"], vp) and torch.equal(out["q"][:n], want["q"][:n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, t, keep_keys=True, out=out, cu_rows=cu)
    for _ in range(3):
        c["kp"].fill_(MARK)
        c["vp"].fill_(MARK)
        out["k"].zero_()
        graph.replay()
        assert torch.equal(c["kp"], kp) and torch.equal(c["vp"], vp) and torch.equal(out["k"][:n], want["k"][:n])


def test_append_refused():
    c = make(27, [5, 0], [3, 4], 4, 2, 64, 16, BF16, behind=0)
    t = sv.RotaryTable(64)
    for kw in (dict(cu_rows=None), dict(kmax=3), dict(cu_drafts=i32([0, 2, 5])), dict(cu_rows=None, kmax=2), dict(cu_rows=i32([0, 3])),
               dict(out={"q": c["q"][:5], "k": None, "status": i32([0, 0])}), dict(out={"q": c["q"], "k": None, "status": i32([0])})):
        with pytest.raises(ValueError):
            call(c, t, **kw)
    with pytest.raises(sv.SpecError):
        call(c, sv.RotaryTable(66))
    with pytest.raises(TypeError):
        sv.spec_cache_append_rotated(c["q"].float(), c["k"], c["v"], c["kp"], c["vp"], c["table"], c["length"], t, cu_rows=i32(c["cu"]))
