"""Workspaces that the cache calls refuse."""

import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


def test_workspaces():
    k = torch.zeros((4, 1, 8, 64), device=DEV)
    q = torch.zeros((1, 2, 64), device=DEV)
    table = i32(1, 4)
    call = lambda out: sv.spec_paged_attention(q, k, k, table, i32(1), None, 0, 1.0, out=out)  # noqa: E731
    good = call(None)
    pool, book = k[None], (i32(1, 4) - 1, i32(1), i32(1), i32(4))
    grow = lambda out: sv.spec_cache_resize(pool, pool.clone(), *book, out=out)  # noqa: E731
    room = grow(None)
    for f, out in ((call, good), (grow, room)):
        ws = out["workspace"]
        wide = torch.zeros(2 * ws.numel(), dtype=torch.uint8, device=DEV)
        for bad in (ws.cpu(), wide[::2]):
            with pytest.raises(TypeError):
                f(dict(out, workspace=bad))
        assert (f(dict(out, workspace=wide.view(torch.int64)))["status"] == 0).all()   # its bytes count
        with pytest.raises(sv.SpecError):
            f(dict(out, workspace=ws[:16]))
