"""Paths of spec_paged_attention that a decode step's usual arguments do not take: other scales, a wait that gave up, batches of
the largest size.  Tolerances as in test_gpu_paged_attention.py."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import cache_reference as ref  # noqa: E402
from tests.test_gpu_paged_attention import call, make, tolerance  # noqa: E402

DEV = "cuda"
# every kernel: bf16 with 64, 128 (80: padded) and 256 columns, float32 up to 128, float32 above
KERNELS = [(64, torch.bfloat16), (80, torch.bfloat16), (128, torch.bfloat16), (256, torch.bfloat16), (64, torch.float32),
           (128, torch.float32), (256, torch.float32)]


@pytest.mark.parametrize("D,dtype", KERNELS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20)])
@pytest.mark.parametrize("scale", ["negative", "zero", "small", "large"])
def test_scales(D, dtype, window, sinks, scale):
    # one stream alone is split over the blocks of threads and joined
    for lengths, drafts in (([0, 130, 311], [2, 5, 0]), ([1203], [3])):
        c = make(30, lengths, drafts, 8, 2, D, 16, dtype)
        c["scale"] = {"negative": -(D ** -0.5), "zero": 0.0, "small": 1e-6, "large": 0.7}[scale]
        got = call(c, window, sinks)
        assert (got["status"] == 0).all()
        to = lambda t: t.float().cpu().numpy()  # noqa: E731
        out, spread = ref.attention(to(c["q"]), to(c["k"]), to(c["v"]), c["table"], c["length"], c["cu"], c["scale"], window, sinks)
        off = np.abs(got["out"].double().cpu().numpy() - out)
        tol = tolerance(dict(c, scale=abs(c["scale"])), out, spread)
        assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("D,dtype", KERNELS)
def test_a_negative_scale_is_a_negated_query(D, dtype):
    c = make(31, [700, 65], [4, 1], 8, 2, D, 16, dtype)
    want = call(dict(c, q=-c["q"]))["out"]
    assert torch.equal(call(dict(c, scale=-c["scale"]))["out"], want)


@pytest.mark.parametrize("D,dtype", KERNELS)
def test_a_wait_that_gave_up_is_reported_until_the_workspace_is_cleared(D, dtype):
    # the word that a wait sets when it gives up, set from the host
    c = make(32, [900, 3, 64], [5, 0, 2], 8, 2, D, 16, dtype)
    out = call(c)
    want = out["out"].clone()
    assert (out["status"] == 0).all()
    out["workspace"][:4].view(torch.int32).fill_(1)
    for _ in range(2):   # it stays
        assert call(c, out=out)["status"].tolist() == [6, 6, 6]
    out["workspace"][:256].zero_()
    call(c, out=out)
    assert out["status"].tolist() == [0, 0, 0] and torch.equal(out["out"], want)


@pytest.mark.parametrize("D,dtype", [(8, torch.bfloat16), (72, torch.bfloat16), (8, torch.float32), (136, torch.float32)])
@pytest.mark.parametrize("B", [5000, 65535])
def test_batches_of_the_largest_size(B, D, dtype):
    # lengths up to 20 and one of 300, appended and attended; the definition for all streams at once in float64
    P, width, Hq = 8, 40, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    length = torch.randint(0, 20, (B,), generator=g, device=DEV, dtype=torch.int32)
    length[B // 3] = 300
    held = (length + P) // P
    ends = torch.cumsum(held, 0)
    pages = int(ends[-1])
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    mine = torch.arange(width, device=DEV)[None] < held[:, None]
    table[mine] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    pool = torch.randn((2, pages, 1, P, D), generator=g, device=DEV).to(dtype)
    new = torch.randn((2, B, 1, D), generator=g, device=DEV).to(dtype)
    q = (2 * torch.randn((B, Hq, D), generator=g, device=DEV)).to(dtype)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    assert (sv.spec_cache_append(new[0], new[1], pool[0], pool[1], table, length, cu, 3, reserved=zero)["status"] == 0).all()
    at = table.long().gather(1, (length // P).long()[:, None])[:, 0]
    for i in range(2):
        assert torch.equal(pool[i][at, 0, (length % P).long()], new[i][:, 0])
    out = sv.spec_paged_attention(q, pool[0], pool[1], table, length, cu, 3, D ** -0.5)
    assert (out["status"] == 0).all()
    got = out["out"].double()
    u, r = 2.0 ** -24, 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    worst = 0.0
    qn, kn = q.double().norm(dim=2).max(), pool[0].double().norm(dim=3).max()
    weight = 0.6932 * (D + 4) * u * 1.4427 * D ** -0.5 * qn * kn + 8 * u + r
    for rows, w in ((torch.arange(B, device=DEV) != B // 3, 3), (torch.arange(B, device=DEV) == B // 3, width)):
        t = table[rows, :w].long().clamp(min=0)
        k, v = (pool[i][t][:, :, 0].reshape(t.shape[0], w * P, D).double() for i in range(2))
        s = torch.einsum("bhd,bnd->bhn", q[rows].double(), k) * D ** -0.5
        seen = torch.arange(w * P, device=DEV)[None] <= length[rows][:, None]
        p = torch.softmax(s.masked_fill(~seen[:, None], float("-inf")), dim=2)
        want = torch.einsum("bhn,bnd->bhd", p, v)
        spread = torch.einsum("bhn,bnd->bhd", p, v.abs()) + want.abs()
        tol = 2 * weight * spread + (340 + 8) * u * (spread + want.abs()) + (r or u) * want.abs() + 1e-30
        worst = max(worst, ((got[rows] - want).abs() / tol).max().item())
    assert worst <= 1, worst
