"""Float32 attention to the last bits: no part of a number, no product of parts and no rounded sum is missing.  Bounds and
their derivation in tests/float32_parts.py."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv
from tests import float32_parts as fp

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def two_keys(inputs, D, seed):
    """The kernel's outputs [n] for a batch of streams with two positions each, the numbers in columns drawn for each."""
    q0, k0, q1, k1, v = (torch.from_numpy(x).to(DEV) for x in inputs)
    n = q0.numel()
    rng = np.random.default_rng(seed)
    cols = torch.from_numpy(np.stack([rng.permutation(D)[:3] for _ in range(n)])).to(DEV)
    at = torch.arange(n, device=DEV)
    q, k, vv = torch.zeros((n, 1, D), device=DEV), torch.zeros((n, 1, 8, D), device=DEV), torch.zeros((n, 1, 8, D), device=DEV)
    q[at, 0, cols[:, 0]], q[at, 0, cols[:, 1]] = q0, q1
    k[at, 0, 0, cols[:, 0]], k[at, 0, 1, cols[:, 1]] = k0, k1
    vv[at, 0, 1, cols[:, 2]] = v
    table = at.to(torch.int32)[:, None].contiguous()
    out = sv.spec_paged_attention(q, k, vv, table, torch.ones(n, dtype=torch.int32, device=DEV), None, 0, 1.0)
    assert (out["status"] == 0).all()
    got = out["out"][:, 0]
    mine = got[at, cols[:, 2]].double().cpu().numpy()
    got[at, cols[:, 2]] = 0
    assert (got == 0).all()
    return mine


@pytest.mark.parametrize("D", [8, 64, 80, 128, 256])
@pytest.mark.parametrize("kind", ["scores", "weights"])
def test_two_keys(kind, D):
    inputs = fp.two_key_inputs(kind, 4096, D)
    want, bound = fp.two_key_output(*inputs)
    got = two_keys(inputs, D, D)
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_value_alone_comes_back(D):
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    n = 500
    pages = torch.randn((2, n, 1, 8, D), generator=g, device=DEV)
    q = torch.randn((n, 1, D), generator=g, device=DEV)
    table = torch.arange(n, dtype=torch.int32, device=DEV)[:, None].contiguous()
    out = sv.spec_paged_attention(q, pages[0], pages[1], table, torch.zeros(n, dtype=torch.int32, device=DEV), None, 0, D ** -0.5)
    v = pages[1][:, :, 0]
    assert ((out["out"] - v).abs() <= 12 * fp.U * v.abs()).all()   # six sums that may be cut off


@pytest.mark.parametrize("D", [64, 128])
def test_sums_over_a_long_context_do_not_drift(D):
    # 160 streams, so that a block of threads adds most of a stream's 79 tiles; positive values, so that cuts add up
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    B, P, n = 160, 64, 5002
    per = -(-(n + 1) // P)
    k = torch.randn((B * per, 1, P, D), generator=g, device=DEV)
    v = 1 + torch.rand((B * per, 1, P, D), generator=g, device=DEV)
    q = torch.randn((B, 1, D), generator=g, device=DEV)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    out = sv.spec_paged_attention(q, k, v, table, torch.full((B,), n, dtype=torch.int32, device=DEV), None, 0, D ** -0.5)
    kk, vv = (x.view(B, per * P, D)[:, :n + 1].double() for x in (k, v))
    w = torch.softmax(torch.einsum("bd,bnd->bn", q[:, 0].double(), kk) * D ** -0.5, dim=1)
    want = torch.einsum("bn,bnd->bd", w, vv)
    shift = ((out["out"][:, 0].double() - want) / want).mean().item()
    assert abs(shift) <= fp.SHIFT, shift


@pytest.mark.parametrize("D", [64, 128, 256])
def test_as_near_as_a_plain_float32_computation(D):
    g = torch.Generator(device=DEV)
    g.manual_seed(7 + D)
    B, P, n = 16, 64, 2000
    per = -(-(n + 1) // P)
    k, v = (torch.randn((B * per, 2, P, D), generator=g, device=DEV) for _ in range(2))
    q = 2.5 * torch.randn((B, 8, D), generator=g, device=DEV)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).view(B, per)
    out = sv.spec_paged_attention(q, k, v, table, torch.full((B,), n, dtype=torch.int32, device=DEV), None, 0, D ** -0.5)

    def plain(dtype):
        kk, vv = (x.view(B, per, 2, P, D).transpose(1, 2).reshape(B, 2, per * P, D)[:, :, :n + 1].to(dtype) for x in (k, v))
        s = torch.matmul(q.view(B, 2, 4, D).to(dtype), kk.transpose(2, 3)) * D ** -0.5
        w = torch.exp(s - s.amax(dim=-1, keepdim=True))
        return (torch.matmul(w, vv) / w.sum(dim=-1, keepdim=True)).reshape(B, 8, D)

    assert not torch.backends.cuda.matmul.allow_tf32
    want = plain(torch.float64)
    off = lambda x: (x.double() - want).square().mean().sqrt().item()  # noqa: E731
    assert off(out["out"]) <= 4 * off(plain(torch.float32)), (off(out["out"]), off(plain(torch.float32)))
