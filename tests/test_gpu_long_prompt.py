"""Prompts of a million tokens: an item's rows see all keys before them, and what waits for the item waits as long as that takes.  A few rows
are compared with the definition in 64 bits."""

import math

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests import prompt_reference as ref  # noqa: E402

DEV = "cuda"


@pytest.mark.parametrize("dtype,n,Hq,D", [(torch.bfloat16, (1 << 20) + 77, 1, 64),    # the last piece has rows of one group alone
                                          (torch.bfloat16, (1 << 19) + 250, 2, 128), (torch.bfloat16, (1 << 18) + 5, 1, 256),
                                          (torch.float32, (1 << 19) + 77, 1, 64)])
def test_long_prompt(dtype, n, Hq, D):
    g = torch.Generator(device=DEV)
    g.manual_seed(61)
    short, scale = 300, D ** -0.5
    x = torch.randn((short + n, Hq + 2, D), generator=g, device=DEV).to(dtype)
    x[:, :Hq] *= 2
    q, k, v = x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:]
    cu = torch.tensor([0, short, short + n], dtype=torch.int32, device=DEV)
    got = sv.spec_prompt_attention(q, k, v, cu, scale)
    assert got["status"].tolist() == [0, 0]
    assert torch.isfinite(got["out"]).all()
    kk, vv = k[short:, 0].double(), v[short:, 0].double()
    for i in [0, 1, 127, 128, 255, 256, 4095, 65536, n // 2, n // 2 + 129, n - 257, n - 256, n - 78, n - 77, n - 2, n - 1]:
        for h in range(Hq):
            s = kk[:i + 1] @ q[short + i, h].double() * scale
            p = torch.softmax(s, dim=0)
            out = p @ vv[:i + 1]
            spread = p @ (vv[:i + 1] - out).abs()
            tol = ref.attention_tolerance(q[short + i:short + i + 1, h:h + 1], k[short:short + i + 1], scale, i + 1, out, spread)
            off = (got["out"][short + i, h].double() - out).abs()
            assert (off <= tol).all(), (i, h, float((off / tol).max()))
    assert not math.isnan(float(got["out"][short - 1].float().sum()))
