"""Float32 attention at the ends of the number range.

u = 2^-24.  A float32 head is computed from three bf16 parts a number: a score's error is at most 15 u |s| (three terms left
out, each below u |s|, and six cut sums of 2 u |s|), a weight's is the scores' plus 4 u, and a sum of two weighted
values' another 21 u (six cut sums, four roundings, the exponential's 2^-22)."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV, U = "cuda", 2.0 ** -24
LARGE = [3.4028234e38, -3.4028234e38, 3.3996e38, 3.396e38, -3.3895314e38, 3.38e38, 1e38, 2.0 ** -126, -1e-37, 0.0]


def attend(q, k, v, scale, window=0):
    """q [B, D], k and v [B, 2, D]: every stream's token sees its own position and the one before."""
    B, _, D = k.shape
    pages = torch.zeros((2, B, 1, 8, D), device=DEV)
    pages[0, :, 0, :2], pages[1, :, 0, :2] = k, v
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].contiguous()
    out = sv.spec_paged_attention(q[:, None].contiguous(), pages[0], pages[1], table, torch.ones(B, dtype=torch.int32, device=DEV), None, 0,
                                  scale, window=window)
    assert (out["status"] == 0).all()
    return out["out"][:, 0].double()


@pytest.mark.parametrize("D", [8, 64, 128, 256])
def test_values(D):
    x = torch.tensor(LARGE, device=DEV)
    v = x[(torch.arange(20, device=DEV)[:, None] + torch.arange(D, device=DEV)) % len(x)][:, None].expand(20, 2, D)
    # a token that sees itself alone: weight 1 (the sum of two such values overflows float32 before its division)
    got = attend(torch.zeros((20, D), device=DEV), torch.zeros((20, 2, D), device=DEV), v, 1.0, window=1)
    want = v[:, 1].double()
    # below the normal numbers the parts are multiples of 2^-133
    assert ((got - want).abs() <= 21 * U * want.abs() + 2.0 ** -131).all()


@pytest.mark.parametrize("D", [8, 64, 128, 256])
@pytest.mark.parametrize("side", ["keys", "queries"])
def test_keys_and_queries(D, side):
    # scores 3.4 and 3.4 x / 3.4028e38 of one column each
    B = D
    col = torch.arange(B, device=DEV)
    q, k, v = torch.zeros((B, D), device=DEV), torch.zeros((B, 2, D), device=DEV), torch.zeros((B, 2, D), device=DEV)
    x = torch.tensor(LARGE, device=DEV)[col % len(LARGE)]
    if side == "keys":
        q[col, col] = 1e-30
        k[col, 0, col], k[col, 1, col] = 3.4028234e38, x
    else:
        q[col, col] = x
        k[col, 0, col], k[col, 1, col] = 1e-30, -0.7e-30
    v[:, 1] = 1.0
    got = attend(q, k, v, 1e-8)
    s = (q.double()[:, None] * k.double()).sum(dim=2) * 1e-8
    p = torch.softmax(s, dim=1)[:, 1:]
    top = s.abs().amax(dim=1, keepdim=True)
    assert ((got - p).abs() <= p * (1 - p) * (30 * top + 8) * U + 21 * U * p).all()


def test_infinities_are_nan_as_documented():
    D = 64
    v = torch.ones((1, 2, D), device=DEV)
    v[0, 1, 3] = float("inf")
    got = attend(torch.zeros((1, D), device=DEV), torch.zeros((1, 2, D), device=DEV), v, 1.0)
    assert torch.isnan(got[0, 3]) and (got[0, :3] == 1).all() and (got[0, 4:] == 1).all()
