"""The one token of a lone stream, turned in place: a single row of a wider projection has that projection's stride, or none."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def wide_row(dtype, Hq=6, Hkv=2, D=64):
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    return torch.randn((1, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("view", [lambda x: x, lambda x: x.reshape(x.shape), lambda x: torch.as_strided(x, x.shape, (384, 64, 1))])
def test_rotate_in_place(view, dtype):
    x = wide_row(dtype)
    t = sv.RotaryTable(64)
    want = sv.spec_rotate(x[:, :6], i32([1234]), t)
    rest = x.clone()
    y = x[:, :6]
    sv.spec_rotate(y, i32([1234]), t, out=view(y))
    assert torch.equal(x[:, :6], want) and torch.equal(x[:, 6:], rest[:, 6:])
    x = rest.clone()
    sv.spec_rotate(view(x[:, :6]), i32([1234]), t, out=x[:, :6])
    assert torch.equal(x[:, :6], want) and torch.equal(x[:, 6:], rest[:, 6:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_in_place(dtype):
    x, t = wide_row(dtype), sv.RotaryTable(64)
    pools = [torch.zeros((3, 2, 16, 64), dtype=dtype, device=DEV) for _ in range(4)]
    table, length = i32([[2, 0]]), i32([17])
    want = sv.spec_cache_append_rotated(x[:, :6], x[:, 6:8], x[:, 8:], pools[0], pools[1], table, length, t, kmax=0, keep_keys=True)
    rest = x.clone()
    got = sv.spec_cache_append_rotated(x[:, :6], x[:, 6:8], x[:, 8:], pools[2], pools[3], table, length, t, kmax=0, keep_keys=True,
                                       out={"q": x[:, :6], "k": x[:, 6:8], "status": i32([99])})
    assert want["status"].tolist() == got["status"].tolist() == [0]
    assert torch.equal(x[:, :6], want["q"]) and torch.equal(x[:, 6:8], want["k"]) and torch.equal(x[:, 8:], rest[:, 8:])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_no_row_in_place():
    x = torch.empty((0, 10, 64), device=DEV)
    assert sv.spec_rotate(x[:, :6], i32([]), sv.RotaryTable(64), out=x[:, :6]).shape == (0, 6, 64)


def test_rows_in_place_still_need_one_stride():
    x = torch.zeros((2, 10, 64), device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_rotate(x[:, :6], i32([0, 1]), sv.RotaryTable(64), out=torch.as_strided(x, (2, 6, 64), (384, 64, 1)))
