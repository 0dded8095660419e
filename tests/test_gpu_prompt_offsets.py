"""The prompt calls where element offsets pass 32 bits: rows, outputs and pools of more than 2^31 elements (tolerances: prompt_reference)."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import prompt_reference as ref  # noqa: E402

DEV = "cuda"


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def noise(shape, seed):
    """Standard normal bf16, the last 4,096 rows of it: what the tests look at.  The others are zero."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    x[-4096:] = torch.randn((4096,) + tuple(shape[1:]), generator=g, device=DEV).to(torch.bfloat16)
    return x


def test_rotate():
    rows = 240000   # x 72 x 128: 2.2e9
    x = noise((rows, 72, 128), 1)
    at = torch.arange(rows, dtype=torch.int32, device=DEV)
    got = sv.spec_rotate(x, at, sv.RotaryTable(128))
    assert not got[0].any()
    want, tol = ref.rotate(x[-64:], at[-64:], ref.frequencies(128))
    assert ((got[-64:].double() - want).abs() <= tol).all()


def test_prompts():
    n, last = 270000, 300   # x 64 x 128: 2.2e9
    q, k, v = noise((n, 64, 128), 2), noise((n, 8, 128), 3), noise((n, 8, 128), 4)
    cu = [0, 100000, 200000, n - last, n]
    got = sv.spec_prompt_attention(q, k, v, i32(cu), 128 ** -0.5, window=64)
    assert (got["status"] == 0).all() and not got["out"][:200000].any()   # zero values
    q, k, v = q[-last:], k[-last:], v[-last:]
    out, spread = ref.attention(q, k, v, [0, last], 128 ** -0.5, 64)
    tol = ref.attention_tolerance(q, k, 128 ** -0.5, last, out, spread)
    assert ((got["out"][-last:].double() - out).abs() <= tol).all()


def test_append():
    pages, P = 17000, 128   # x 8 x 128 x 128: 2.2e9
    pools = [torch.zeros((pages, 8, P, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q, k, v = (noise((4096, h, 128), 5 + h)[:200] for h in (16, 8, 8))
    table = i32([[pages - 1, pages - 3, pages - 2]])
    got = sv.spec_cache_append_rotated(q, k, v, *pools, table, i32([100]), sv.RotaryTable(128), cu_rows=i32([0, 200]), keep_keys=True)
    assert got["status"].tolist() == [0]
    at = torch.arange(100, 300, device=DEV)
    want, tol = ref.rotate(k, at, ref.frequencies(128))
    page = table[0].long()[at // P]
    assert ((pools[0][page, :, at % P].double() - want).abs() <= tol).all() and torch.equal(pools[1][page, :, at % P], v)
    for pool in pools:
        for b in range(0, pages - 3, 1700):
            assert not pool[b:min(b + 1700, pages - 3)].any()
    want, tol = ref.rotate(q, at, ref.frequencies(128))
    assert ((got["q"].double() - want).abs() <= tol).all()
