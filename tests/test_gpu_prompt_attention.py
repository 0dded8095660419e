"""spec_prompt_attention against the definition in 64 bits (tolerances: prompt_reference)."""

import math

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


def make(seed, rows, Hq, Hkv, D, dtype=BF16, behind=3, gain=2.0):
    """Slices of one projection; `behind` rows of NaN and infinities follow the last prompt."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = sum(rows)
    wide = torch.randn((n + behind, Hq + 2 * Hkv, D), generator=g, device=DEV)
    wide[:, :Hq] *= gain
    if behind:
        wide[n:] = math.nan
        wide[n + 1:] = math.inf
    wide = wide.to(dtype)
    cu = [0] + list(np.cumsum(rows))
    return dict(q=wide[:, :Hq], k=wide[:, Hq:Hq + Hkv], v=wide[:, Hq + Hkv:], cu=cu, scale=D ** -0.5, rows=rows,
                d_cu=torch.tensor(cu, dtype=torch.int32, device=DEV))


def call(c, window=0, sinks=0, scale=None, out=None, stream=None):
    return sv.spec_prompt_attention(c["q"], c["k"], c["v"], c["d_cu"], c["scale"] if scale is None else scale, window=window, sinks=sinks, out=out,
                                    stream=stream)


def check(c, window=0, sinks=0, scale=None, got=None):
    scale = c["scale"] if scale is None else scale
    if got is None:
        n = c["q"].shape[0]
        mark = torch.full(c["q"].shape, -77.0, dtype=c["q"].dtype, device=DEV)
        got = call(c, window, sinks, scale, out={"out": mark, "status": torch.full((len(c["rows"]),), 99, dtype=torch.int32, device=DEV)})
        assert (got["out"][c["cu"][-1]:n] == -77).all()   # rows behind the last prompt
    assert (got["status"] == 0).all()
    n = c["cu"][-1]
    q, k, v = c["q"][:n], c["k"][:n], c["v"][:n]
    out, spread = ref.attention(q, k, v, c["cu"], scale, window, sinks)
    tol = ref.attention_tolerance(q, k, scale, max(c["rows"]) if c["rows"] else 0, out, spread)
    off = (got["out"][:n].double() - out).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (float((off / tol).nan_to_num(nan=math.inf).max()), bad.nonzero()[:4].tolist(), int(bad.sum()))


HEADS = [(1, 1, 64), (4, 4, 64), (7, 1, 128), (16, 4, 64), (24, 8, 128), (64, 8, 128), (128, 1, 64), (6, 2, 128), (10, 2, 80), (3, 1, 96), (8, 2, 8),
         (8, 1, 120)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_heads(Hq, Hkv, D, dtype):
    check(make(1, [1, 0, 5, 130, 300, 0], Hq, Hkv, D, dtype))


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 256), (8, 1, 256), (12, 4, 136), (6, 2, 192), (64, 2, 200)])
def test_wide_heads(Hq, Hkv, D):
    check(make(2, [1, 63, 64, 65, 300, 0, 17], Hq, Hkv, D))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (14, 2)])
def test_lengths_around_tiles_and_pieces(Hq, Hkv, dtype):
    check(make(3, [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 383, 384, 385, 511, 513], Hq, Hkv, 64, dtype))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 200), (5, 0), (63, 3), (64, 64), (65, 1), (127, 0), (128, 129), (129, 4), (200, 300),
                                          (500, 16), (5000, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_window_and_sinks(window, sinks, dtype):
    check(make(4, [700, 3, 129, 0, 600], 8, 2, 64, dtype), window, sinks)


@pytest.mark.parametrize("window,sinks", [(100, 4), (300, 0), (1, 70)])
def test_window_of_wide_and_single_heads(window, sinks):
    check(make(5, [700, 90], 4, 2, 256), window, sinks)
    check(make(5, [700, 90], 2, 2, 128), window, sinks)
    check(make(5, [700, 90], 7, 1, 128), window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-20, 1.5])
def test_scales(scale, dtype):
    check(make(6, [40, 200], 4, 2, 64, dtype), scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_that_keep_rising_and_falling(dtype):
    # the running maximum is raised tile after tile; and one early key carries everything
    c = make(7, [900], 2, 1, 64, dtype, behind=0)
    up = torch.linspace(0.1, 3.0, 900, device=DEV)[:, None, None]
    c["q"].copy_(torch.ones_like(c["q"]) * 3)
    c["k"].copy_((up * torch.ones_like(c["k"])).to(dtype))
    check(c)
    c["k"].copy_((up.flip(0) * torch.ones_like(c["k"])).to(dtype))
    check(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long(dtype):
    check(make(8, [3000, 1, 2111], 4, 1, 128, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B", [33, 256, 257, 700])
def test_many_prompts(B, dtype):
    rng = np.random.default_rng(B)
    check(make(9, rng.integers(0, 40, B).tolist(), 4, 2, 64, dtype))


def test_very_many_prompts():
    rows = [1] * 65535
    rows[100], rows[65534], rows[0] = 0, 5, 2
    c = make(10, rows, 2, 1, 8)
    got = call(c)
    assert (got["status"] == 0).all()
    cu = np.array(c["cu"])
    ones = torch.from_numpy(cu[:-1][np.array(rows) == 1]).to(DEV)
    assert torch.equal(got["out"][ones], c["v"][ones].expand(-1, 2, -1))   # a token alone sees itself
    last = dict(c, q=c["q"][cu[-2]:cu[-1]], k=c["k"][cu[-2]:cu[-1]], v=c["v"][cu[-2]:cu[-1]], cu=[0, 5], rows=[5])
    check(last, got={"out": got["out"][cu[-2]:cu[-1]], "status": got["status"]})


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_prompt_without_offsets(dtype):
    c = make(11, [333], 4, 2, 64, dtype, behind=0)
    check(c, got=sv.spec_prompt_attention(c["q"], c["k"], c["v"], None, c["scale"]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_of_another_prompt_is_seen(dtype):
    rows = [70, 130, 1, 200, 64, 333]
    c = make(12, rows, 8, 2, 64, dtype)
    for b in (1, 3, 4):   # keys and values of these are not finite
        c["k"][c["cu"][b]:c["cu"][b + 1]] = math.nan
        c["v"][c["cu"][b]:c["cu"][b + 1]] = math.inf
    got = call(c)
    for b in (0, 2, 5):
        s = slice(c["cu"][b], c["cu"][b + 1])
        one = dict(c, q=c["q"][s], k=c["k"][s], v=c["v"][s], cu=[0, rows[b]], rows=[rows[b]])
        check(one, got={"out": got["out"][s], "status": got["status"]})


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_no_row_sees(dtype):
    # with a window, what has left it for every row of the prompt's end no longer counts, whatever it is
    c = make(13, [600], 8, 2, 64, dtype)
    got0 = call(c, window=100, sinks=2)["out"].clone()
    c["v"][5:10] = math.nan
    c["k"][5:10] = math.nan
    got = call(c, window=100, sinks=2)["out"]
    assert torch.equal(got[400:600], got0[400:600])
    assert not torch.isfinite(got[5:10].float()).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_what_is_not_finite(dtype):
    c = make(14, [300], 2, 1, 64, dtype)
    c["v"][20, 0, 3] = math.nan
    got = call(c)["out"].float()
    assert torch.isnan(got[20:300, :, 3]).all()
    keep = torch.ones(64, dtype=torch.bool, device=DEV)
    keep[3] = False
    assert torch.isfinite(got[:300][:, :, keep]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu,first", [([1, 5, 9], 0), ([0, 5, 4], 1), ([0, 5, 13], 1), ([0, 300, 400], 0), ([0, 5, 3, 9, 12], 1), ([-4, 5, 9], 0)])
def test_broken_offsets(cu, first, dtype):
    c = make(15, [5, 4, 3], 4, 2, 64, dtype, behind=0)   # 12 rows
    mark = torch.full(c["q"].shape, -77.0, dtype=dtype, device=DEV)
    got = sv.spec_prompt_attention(c["q"], c["k"], c["v"], torch.tensor(cu, dtype=torch.int32, device=DEV), c["scale"],
                                   out={"out": mark, "status": torch.zeros(len(cu) - 1, dtype=torch.int32, device=DEV)})
    assert got["status"].tolist() == [0 if b < first else 5 for b in range(len(cu) - 1)]
    n = cu[first] if first else 0
    assert (got["out"][n:] == -77).all()
    if first:
        one = dict(c, q=c["q"][:n], k=c["k"][:n], v=c["v"][:n], cu=[0, n], rows=[n])
        check(one, got={"out": got["out"][:n], "status": got["status"][:1]})


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broken_offsets_behind_many(dtype):
    rows = [3] * 600
    c = make(16, rows, 2, 1, 64, dtype, behind=0)
    cu = list(c["cu"])
    cu[401] = 2   # prompt 400 has a negative count
    got = sv.spec_prompt_attention(c["q"], c["k"], c["v"], torch.tensor(cu, dtype=torch.int32, device=DEV), c["scale"])
    assert got["status"].tolist() == [0] * 400 + [5] * 200


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_rows(dtype):
    e = torch.empty((0, 4, 64), dtype=dtype, device=DEV)
    got = sv.spec_prompt_attention(e, e[:, :2], e[:, :2], torch.zeros(4, dtype=torch.int32, device=DEV), 0.1)
    assert got["status"].tolist() == [0, 0, 0] and got["out"].shape == (0, 4, 64)
    got = sv.spec_prompt_attention(e, e[:, :2], e[:, :2], torch.tensor([0, 0, 1], dtype=torch.int32, device=DEV), 0.1)
    assert got["status"].tolist() == [0, 5]
    got = sv.spec_prompt_attention(e, e[:, :2], e[:, :2], torch.zeros(1, dtype=torch.int32, device=DEV), 0.1)
    assert got["status"].shape == (0,)
    x = torch.ones((3, 4, 64), dtype=dtype, device=DEV)   # rows, and prompts without any
    got = sv.spec_prompt_attention(x, x[:, :2], x[:, :2], torch.zeros(4, dtype=torch.int32, device=DEV), 0.1)
    assert got["status"].tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_same_bits_on_another_stream_and_replayed(dtype):
    c = make(17, [400, 37, 1500, 0, 222], 16, 4, 128, dtype)
    n = c["cu"][-1]
    want = call(c)["out"][:n].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = call(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out["out"][:n], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out=out)
    for _ in range(3):
        out["out"].zero_()
        graph.replay()
        assert torch.equal(out["out"][:n], want)
    # two at once, each with its own outputs
    outs = [call(c), call(c)]
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        call(c, out=outs[0])
        call(c, out=outs[1], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for o in outs:
            assert torch.equal(o["out"][:n], want)
            o["out"].zero_()


def test_dense_and_sliced_rows_agree():
    c = make(18, [100, 50], 8, 2, 64, behind=0)
    d = dict(c, q=c["q"].contiguous(), k=c["k"].contiguous(), v=c["v"].contiguous())
    assert torch.equal(call(c)["out"], call(d)["out"])


def test_binding_refuses():
    c = make(19, [20], 8, 2, 64, behind=0)
    q, k, v, cu = c["q"], c["k"], c["v"], c["d_cu"]
    f = sv.spec_prompt_attention
    for args, what in [((q.cpu(), k, v, cu, 0.1), TypeError), ((q, k.float(), v, cu, 0.1), TypeError), ((q.half(), k.half(), v.half(), cu, 0.1), TypeError),
                       ((q, k[:19], v, cu, 0.1), ValueError), ((q, k, v, cu.long(), 0.1), TypeError), ((q, k, v[:, :1], cu, 0.1), ValueError),
                       ((q.transpose(0, 1), k, v, cu, 0.1), ValueError), ((q, k, v, cu.cpu(), 0.1), TypeError), ((q[:, :7], k, v, cu, 0.1), sv.SpecError),
                       ((q, k, v, cu[:0], 0.1), ValueError)]:
        with pytest.raises(what):
            f(*args)
    odd = torch.zeros(20 * 12 * 64 + 1, dtype=BF16, device=DEV)[1:].view(20, 12, 64)
    with pytest.raises(sv.SpecError):   # not on 16-byte boundaries
        f(odd[:, :8], odd[:, 8:10], odd[:, 10:], cu, 0.1)
    wide = torch.zeros((20, 2, 136), dtype=F32, device=DEV)
    with pytest.raises(sv.SpecError):   # float32 heads above 128
        f(wide, wide, wide, cu, 0.1)
    with pytest.raises(ValueError):
        f(q, k, v, cu, 0.1, out={"out": torch.empty((19, 8, 64), dtype=BF16, device=DEV), "status": torch.empty(1, dtype=torch.int32, device=DEV)})
