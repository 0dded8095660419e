"""spec_paged_attention and spec_cache_append against plain float64 definitions.

Tolerances, from the arithmetic alone (u = 2^-24 float32; r = 2^-8: a bf16
significand has 8 bits, so rounding to nearest moves a value by at most 2^-8 of it):
* a score in base 2 is a float32 dot product of D terms and one multiplication, so its error is at
  most e_s = (D + 4) u log2(e) scale max|q|_2 |k|_2 (Cauchy-Schwarz), and a weight's relative error ln 2
  e_s + 4 u (exp2, rescalings) + r with bf16 weights;
* a relative error d of the weights moves the output by at most 2 d spread (spread = sum p |v - out|);
* the values' sum adds (positions + 8) u sum p |v|, and the output's rounding r |out| in bf16.
"""

import ctypes

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def tolerance(c, out, spread):
    u, r = 2.0 ** -24, 2.0 ** -8
    D, bf16 = c["q"].shape[2], c["q"].dtype == torch.bfloat16
    qn = c["q"].double().norm(dim=2).max().item()
    kn = c["k_seen"]
    es = (D + 4) * u * 1.4427 * c["scale"] * qn * kn
    d = 0.6932 * es + 4 * u * (1 + max(c["length"]) / 64) + (r if bf16 else 0.0)
    biggest = max(c["length"]) + 40
    return 2 * d * spread + (biggest + 8) * u * (spread + np.abs(out)) + (r if bf16 else u) * np.abs(out) + 1e-30


def make(seed, lengths, drafts, Hq, Hkv, D, P, dtype=torch.bfloat16, poison=True, spare=5, q_gain=2.0, kmax=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(lengths)
    need = [-(-(n + d + 1) // P) for n, d in zip(lengths, drafts)]
    width = max(need) + 2
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    k = torch.randn((pages, Hkv, P, D), generator=g, device=DEV).to(dtype)
    v = torch.randn((pages, Hkv, P, D), generator=g, device=DEV).to(dtype)
    kn = k.double().norm(dim=3).max().item()
    if poison:   # slots past a block's end, and pages of nobody
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV)
        for pool in (k, v):
            fill = bad[torch.randint(0, 3, (pages, 1, P, 1), generator=g, device=DEV)].to(dtype)
            keep = torch.zeros((pages, 1, P, 1), dtype=torch.bool, device=DEV)
            for b in range(B):
                n = lengths[b] + drafts[b] + 1
                pos = torch.arange(n, device=DEV)
                keep[torch.from_numpy(table[b]).to(DEV).long()[pos // P], 0, pos % P, 0] = True
            pool.copy_(torch.where(keep, pool, fill))
    cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    q = (q_gain * torch.randn((int(cu[-1]) + B, Hq, D), generator=g, device=DEV)).to(dtype)
    return dict(q=q, k=k, v=v, table=table, length=list(lengths), cu=cu, scale=D ** -0.5,
                kmax=max(drafts) if kmax is None else kmax, k_seen=kn,
                d_table=torch.from_numpy(table).to(DEV), d_len=torch.tensor(lengths, dtype=torch.int32, device=DEV),
                d_cu=torch.from_numpy(cu).to(DEV))


def call(c, window=0, sinks=0, out=None, q=None, cu="own", stream=None):
    return sv.spec_paged_attention(c["q"] if q is None else q, c["k"], c["v"], c["d_table"], c["d_len"],
                                   c["d_cu"] if isinstance(cu, str) else cu, c["kmax"], c["scale"], window=window,
                                   sinks=sinks, out=out, stream=stream)


def check(c, window=0, sinks=0, got=None):
    got = call(c, window, sinks) if got is None else got
    to = lambda t: t.float().cpu().numpy()  # noqa: E731
    out, spread = ref.attention(to(c["q"]), to(c["k"]), to(c["v"]), c["table"], c["length"], c["cu"], c["scale"], window, sinks)
    g = got["out"].double().cpu().numpy()
    assert (got["status"] == 0).all()
    off = np.abs(g - out)
    tol = tolerance(c, out, spread)
    assert np.isfinite(g).all()
    assert (off <= tol).all(), (float((off / tol).max()), np.argwhere(off > tol)[:4])


HEADS = [(1, 1, 64), (4, 4, 64), (7, 1, 128), (16, 4, 64), (24, 8, 128), (64, 8, 128), (32, 1, 128), (10, 2, 80), (8, 2, 8),
         (8, 2, 256), (12, 4, 136)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_heads(Hq, Hkv, D, dtype):
    check(make(1, [0, 5, 64, 130, 311], [3, 0, 5, 2, 4], Hq, Hkv, D, 16, dtype))


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_page_sizes_and_edges(P, dtype):
    # blocks that end before, on and after a page's and a tile's edge
    lengths = [0, 1, P - 6, P - 5, P - 1, P, P + 1, 57, 58, 59, 63, 64, 65, 2 * P + 3, 127, 128, 255]
    check(make(2, lengths, [5] * len(lengths), 8, 2, 64, P, dtype))


@pytest.mark.parametrize("kmax", [0, 1, 9, 15, 16, 31, 32])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (16, 2), (15, 3), (64, 1)])
def test_block_lengths(kmax, Hq, Hkv):
    check(make(3, [0, 100, 77], [kmax, kmax // 2, 0], Hq, Hkv, 128, 16, kmax=kmax))


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (6, 64), (63, 0), (64, 65), (65, 4), (100, 200), (200, 1), (500, 16),
                                          (5000, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_window_and_sinks(window, sinks, dtype):
    check(make(4, [0, 3, 60, 64, 199, 640, 1000], [5, 4, 5, 0, 5, 3, 5], 8, 2, 64, 16, dtype), window, sinks)


def test_pages_outside_the_window_are_not_needed():
    c = make(5, [1000, 333], [5, 2], 8, 2, 128, 16)
    window, sinks = 100, 20
    expected = call(c, window, sinks)["out"].clone()
    for b, n in enumerate(c["length"]):
        first, last = -(-sinks // 16), (n + 1 - window) // 16
        c["k"][c["d_table"][b, first:last].long()] = float("nan")
        c["v"][c["d_table"][b, first:last].long()] = float("inf")
        c["d_table"][b, first:last] = -1
    got = call(c, window, sinks)
    assert (got["status"] == 0).all() and torch.equal(got["out"], expected)
    # the page that the window begins in: its positions before the window may hold anything
    low = c["length"][0] + 1 - window
    page = int(c["d_table"][0, low // 16])
    c["v"][page, :, :low % 16] = float("nan")
    c["k"][page, :, :low % 16] = float("inf")
    assert torch.equal(call(c, window, sinks)["out"], expected)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(64, 8, 128, torch.bfloat16), (16, 2, 64, torch.bfloat16), (8, 2, 128, torch.float32),
                                            (4, 1, 256, torch.bfloat16)])
def test_long_context_is_split_and_joined(Hq, Hkv, D, dtype):
    check(make(6, [5003], [3], Hq, Hkv, D, 32, dtype))


def test_many_short_streams():
    rng = np.random.default_rng(0)
    check(make(7, [int(x) for x in rng.integers(0, 90, 700)], [int(x) for x in rng.integers(0, 3, 700)], 4, 2, 64, 8))


@pytest.mark.parametrize("D", [128, 64, 72])
def test_many_short_streams_in_float32(D):
    # items of one to five tiles, several to a CTA: keys are split two tiles ahead of values, into the next items
    rng = np.random.default_rng(1)
    lengths = [int(x) for x in rng.integers(0, 310, 230)]
    check(make(23, lengths, [int(x) for x in rng.integers(0, 4, 230)], 6, 3, D, 16, torch.float32))


@pytest.mark.parametrize("Hq,kmax", [(1, 7), (9, 0), (1, 15), (17, 0), (32, 0), (11, 2), (8, 5), (7, 6), (8, 7), (13, 4), (8, 8), (8, 9),
                                     (8, 32)])
@pytest.mark.parametrize("D", [144, 256])
def test_rows_of_wide_float32_heads(Hq, kmax, D):
    # 8 to 264 rows a key head: every number of rows a group can have, and groups that are not full
    check(make(24, [70, 0, 333], [kmax, 0, kmax // 2], Hq, 1, D, 32, torch.float32, kmax=kmax))


def test_scores_far_apart():
    # one key carries the row, then another: the running maximum moves by hundreds
    c = make(8, [700], [2], 4, 1, 64, 16, q_gain=40.0)
    check(c)


def test_equal_keys_and_values():
    c = make(9, [300, 17], [4, 1], 8, 2, 128, 16, poison=False)
    c["k"].zero_()
    c["v"].fill_(3.0)
    got = call(c)["out"]
    assert torch.equal(got, torch.full_like(got, 3.0))


def test_infinite_scores_and_values():
    # a visible key of -inf score has no weight; NaN and +inf reach exactly the rows that see them
    c = make(10, [70], [3], 4, 1, 64, 16, poison=False)
    c["q"][:, :, 0] = 1.0
    page, slot = int(c["table"][0, 10 // 16]), 10 % 16
    c["k"][page, 0, slot] = 0.0
    c["k"][page, 0, slot, 0] = float("-inf")
    got = call(c)["out"]
    assert torch.isfinite(got).all()
    seen = c["k"].clone()
    seen[page, 0, slot, 0] = -1e30 if c["k"].dtype == torch.float32 else -3e38
    c["k"] = seen
    assert torch.equal(call(c)["out"], got)
    c["v"][page, 0, slot + 1, 5] = float("inf")
    got = call(c)["out"]
    assert torch.isinf(got[:, :, 5]).all() and torch.isfinite(got[:, :, :5]).all() and torch.isfinite(got[:, :, 6:]).all()
    c["k"][page, 0, slot + 2, 0] = float("nan")
    assert torch.isnan(call(c)["out"]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,extra", [(0, 24), (0, 3), (1, 0), (2, 5), (8, 8)])
def test_rows_of_a_wider_projection(dtype, offset, extra):
    c = make(11, [40, 90], [3, 5], 8, 2, 64, 16, dtype)
    rows, Hq, D = c["q"].shape
    wide = torch.full((rows * (Hq * D + extra) + offset + 64,), float("nan"), dtype=dtype, device=DEV)
    q = torch.as_strided(wide, (rows, Hq, D), (Hq * D + extra, D, 1), offset)
    q.copy_(c["q"])
    check(c, got=call(c, q=q))


def test_dense_blocks_without_offsets():
    c = make(12, [100, 3, 64], [0, 0, 0], 16, 4, 64, 16)
    assert torch.equal(call(c, cu=None)["out"], call(c)["out"])
    c = make(13, [100, 3, 64], [4, 4, 4], 16, 4, 64, 16)
    assert torch.equal(call(c, cu=None)["out"], call(c)["out"])


def test_runs_are_equal_and_workspaces_can_be_shared():
    a = make(14, [3000, 100, 900], [5, 2, 4], 64, 8, 128, 16)
    b = make(15, [50, 60], [1, 0], 64, 8, 128, 16)
    first = call(a)
    want = first["out"].clone()
    alone = call(b)["out"].clone()
    for _ in range(3):
        other = {"out": torch.empty_like(b["q"]), "status": torch.empty(2, dtype=torch.int32, device=DEV),
                 "workspace": first["workspace"]}
        assert torch.equal(call(b, out=other)["out"], alone)
        first["out"].zero_()
        first["workspace"][256:].fill_(255)
        assert torch.equal(call(a, out=first)["out"], want)


def test_another_stream_and_a_graph():
    c = make(16, [500, 1200], [5, 5], 32, 8, 128, 16)
    want = call(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(c, stream=side)
    side.synchronize()
    assert torch.equal(got["out"], want["out"])
    out = call(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out=out)
    # lengths are read when the graph runs: the block moves back by one position
    c["d_len"] -= 1
    graph.replay()
    torch.cuda.synchronize()
    c["length"] = [n - 1 for n in c["length"]]
    assert torch.equal(out["out"], call(c)["out"])


def test_large_pool_offsets():
    # page 300,000 lies past 2^31 elements and past 4 GiB
    P, Hkv, D = 16, 4, 128
    pages = 300001
    k = torch.empty((pages, Hkv, P, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty((pages, Hkv, P, D), dtype=torch.bfloat16, device=DEV)
    c = make(17, [130], [2], 8, Hkv, D, P, poison=False)
    far = torch.arange(pages - 9, pages, device=DEV)
    near = c["d_table"][0, :9].long()
    k[far], v[far] = c["k"][near], c["v"][near]
    want = call(c)["out"]
    c["k"], c["v"] = k, v
    c["d_table"][0, :9] = far.to(torch.int32)
    assert torch.equal(call(c)["out"], want)
    nk = torch.randn((3, Hkv, D), device=DEV).to(torch.bfloat16)
    assert (sv.spec_cache_append(nk, nk, k, v, c["d_table"], c["d_len"], c["d_cu"], 2)["status"] == 0).all()
    for i in range(3):
        assert torch.equal(k[far[(130 + i) // P], :, (130 + i) % P], nk[i])


def test_statuses():
    c = make(18, [40, 50, 60, 70], [2, 2, 2, 2], 8, 2, 64, 16)
    want = call(c)["out"].clone()
    c["d_len"][1] = -1
    got = call(c)
    assert got["status"].tolist() == [0, 9, 0, 0]
    keep = torch.ones(12, dtype=torch.bool, device=DEV)
    keep[3:6] = False
    assert torch.equal(got["out"][keep], want[keep]) and torch.isnan(got["out"][~keep].float()).all()
    c["d_len"][1] = c["d_table"].shape[1] * 16 - 2
    assert call(c)["status"].tolist() == [0, 9, 0, 0]
    c["d_len"][1] = 50
    c["d_table"][2, 1] = c["k"].shape[0]
    got = call(c)
    assert got["status"].tolist() == [0, 0, 10, 0]
    assert torch.equal(got["out"][:6], want[:6]) and torch.equal(got["out"][9:], want[9:])
    assert torch.isfinite(got["out"].float()).all()
    c["d_table"][2, 1] = int(c["table"][2, 1])
    c["d_cu"][2] = 100
    got = call(c)
    assert got["status"].tolist() == [0, 5, 5, 5]
    assert torch.equal(got["out"][:3], want[:3])
    c["d_cu"][2] = 4
    c["d_cu"][0] = 1
    assert call(c)["status"].tolist() == [5, 5, 5, 5]


def test_empty_batch():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    out = sv.spec_paged_attention(torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV), k, k, i32(0, 3), i32(0), i32(1), 3, 1.0)
    assert out["out"].shape == (0, 4, 64)
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    sv.spec_cache_append(none, none, k, k, i32(0, 3), i32(0), i32(1), 3)


def test_refusals():
    c = make(19, [40], [2], 8, 2, 64, 16)
    i32 = c["d_len"]
    with pytest.raises(TypeError):
        sv.spec_paged_attention(c["q"].float(), c["k"], c["v"], c["d_table"], i32, c["d_cu"], 2, 1.0)
    with pytest.raises(TypeError):
        sv.spec_paged_attention(c["q"].cpu(), c["k"], c["v"], c["d_table"], i32, c["d_cu"], 2, 1.0)
    with pytest.raises(TypeError):
        sv.spec_paged_attention(c["q"].half(), c["k"].half(), c["v"].half(), c["d_table"], i32, c["d_cu"], 2, 1.0)
    with pytest.raises(TypeError):
        call(dict(c, d_len=i32.long()))
    with pytest.raises(ValueError):
        call(dict(c, q=c["q"][:, :7]))
    with pytest.raises(ValueError):
        call(dict(c, q=c["q"].transpose(0, 1)))
    with pytest.raises(ValueError):
        call(dict(c, k=c["k"].transpose(1, 2)))
    with pytest.raises(ValueError):
        call(c, cu=None, q=c["q"][:2])
    for bad in (dict(kmax=33), dict(kmax=-1), dict(scale=float("inf"))):
        with pytest.raises(sv.SpecError):
            call(dict(c, **bad))
    with pytest.raises(sv.SpecError):
        call(c, window=-1)
    short = call(c)
    short["workspace"] = short["workspace"][:256]
    with pytest.raises(sv.SpecError) as e:
        call(c, out=short)
    assert e.value.code == -6
    odd = torch.zeros(c["k"].shape[:2] + (12, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(c["q"], odd, odd, c["d_table"], i32, c["d_cu"], 2, 1.0)
    flat = torch.zeros(c["k"].numel() + 1, dtype=torch.bfloat16, device=DEV)[1:].view(c["k"].shape)
    with pytest.raises(sv.SpecError):
        call(dict(c, k=flat))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,D,P", [(1, 64, 8), (8, 128, 16), (3, 80, 64), (2, 8, 256)])
@pytest.mark.parametrize("offset,extra", [(0, 0), (0, 16), (1, 3)])
def test_append(dtype, Hkv, D, P, offset, extra):
    lengths, drafts = [0, 7, P - 1, P, 100], [5, 0, 5, 32, 3]
    c = make(20, lengths, drafts, Hkv, Hkv, D, P, dtype, poison=False)
    rows = int(c["cu"][-1]) + len(lengths)
    wide = torch.randn(2, rows * (Hkv * D + extra) + offset + 8, device=DEV).to(dtype)
    k, v = (torch.as_strided(w, (rows, Hkv, D), (Hkv * D + extra, D, 1), w.storage_offset() + offset) for w in wide)
    ek, ev = c["k"].clone(), c["v"].clone()
    for b in range(len(lengths)):
        for i in range(drafts[b] + 1):
            p, r = lengths[b] + i, int(c["cu"][b]) + b + i
            ek[int(c["table"][b, p // P]), :, p % P] = k[r]
            ev[int(c["table"][b, p // P]), :, p % P] = v[r]
    got = sv.spec_cache_append(k, v, c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], c["kmax"])
    assert (got["status"] == 0).all()
    assert torch.equal(c["k"], ek) and torch.equal(c["v"], ev)


def test_append_statuses():
    c = make(21, [10, 20, 30, 40], [3, 3, 3, 3], 2, 2, 64, 16, poison=False)
    k = torch.randn((16, 2, 64), device=DEV).to(torch.bfloat16)
    before = c["k"].clone()
    c["d_len"][0] = -5
    c["d_table"][1, 1] = -1
    c["d_cu"][3] = 5
    got = sv.spec_cache_append(k, k, c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], 3)
    assert got["status"].tolist() == [9, 10, 5, 5]
    assert torch.equal(c["k"], before)   # stream 1's rows all lie in the page that is not there
    with pytest.raises(sv.SpecError):
        sv.spec_cache_append(k, k, c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], 33)
    with pytest.raises(TypeError):
        sv.spec_cache_append(k.float(), k, c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], 3)
    with pytest.raises(ValueError):
        sv.spec_cache_append(k, k[:3], c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], 3)


def test_append_then_attend():
    c = make(22, [33, 200], [5, 2], 8, 2, 128, 16)
    rows = c["q"].shape[0]
    k, v = (torch.randn((rows, 2, 128), device=DEV).to(torch.bfloat16) for _ in range(2))
    sv.spec_cache_append(k, v, c["k"], c["v"], c["d_table"], c["d_len"], c["d_cu"], c["kmax"])
    check(c)


def test_c_entry_errors():
    L = sv.lib()
    assert L.spec_paged_attention(None, None) == -1 and L.spec_cache_append(None, None) == -1
    assert L.spec_paged_attention_workspace_bytes(None) == 0
    z = (ctypes.c_char * 144)()
    assert L.spec_paged_attention(z, None) == -3   # all sizes zero
