"""A serving loop's life over a pool that is too small for it: whatever fits, every kept token of every stream is in the
cache as it was written, and nobody else's."""

import numpy as np
import pytest

import speculative_decoding_block_verify_gb300 as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = "cuda"


# the last column: whether a holder is passed over because a waiting one has more tokens in its page (known from the
# page model, as is that every pool runs out)
@pytest.mark.parametrize("B,pages,P,seed,longer", [(4, 9, 8, 0, False), (4, 5, 8, 7, True), (8, 9, 16, 7, True), (8, 10, 8, 5, True),
                                                   (40, 44, 8, 6, True), (40, 44, 16, 5, True), (300, 310, 8, 2, True)])
def test_kept_tokens_stay_as_they_were_written(B, pages, P, seed, longer):
    rng = np.random.default_rng(seed)
    kmax, width = 5, 12
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    d = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    k = torch.zeros((2, pages, 1, P, 8), device=DEV)
    v = torch.zeros_like(k)
    book = (table, held, length, refs) = (i32(B, width) - 1, i32(B), i32(B), i32(pages))
    tokens = [[] for _ in range(B)]   # what each stream has kept
    serial, waited, passed = 1, 0, 0
    for step in range(60):
        n = rng.integers(0, kmax + 1, B)   # drafts
        back = np.array([-min(len(t), int(rng.integers(0, 2 * P))) if rng.random() < 0.15 else 0 for t in tokens])
        gone = rng.random(B) < (0.02 if longer else 0.06)
        back[gone] = [-len(tokens[b]) for b in np.flatnonzero(gone)]
        room = np.where(rng.random(B) < 0.1, 0, n + 1)
        reserved = sv.spec_cache_resize(k, v, *book, advance=d(back), room=d(room))["status"]
        r = reserved.tolist()
        for b in range(B):
            if r[b] != 9:   # 9: the row is too short for the block, and the stream is left as it was
                tokens[b] = tokens[b][:len(tokens[b]) + int(back[b])]
        assert set(r) <= {0, 8, 9}
        cu = d(np.concatenate([[0], np.cumsum(n)]))
        rows = int(n.sum()) + B
        new = torch.arange(serial, serial + rows, dtype=torch.float32, device=DEV)
        first = np.concatenate([[0], np.cumsum(n + 1)[:-1]]) + serial
        serial += rows
        # a stream that asked for no room has no block: it is passed over like those that got none
        ask = torch.where(d(room) > 0, reserved, 9)
        for layer in range(2):
            x = (new + 0.25 * layer)[:, None, None].expand(rows, 1, 8).contiguous()
            st = sv.spec_cache_append(x, -x, k[layer], v[layer], table, length, cu, kmax, reserved=ask.to(torch.int32))["status"].tolist()
        kept = np.zeros(B, np.int64)
        for b in range(B):
            assert st[b] in (0, 8, 9) and (st[b] == 0 or room[b] == 0 or r[b] != 0 or st[b] == 8)
            waited += r[b] == 8
            passed += r[b] == 0 and room[b] > 0 and st[b] == 8
            if st[b] == 0:
                kept[b] = rng.integers(0, n[b] + 2)
                tokens[b] += [int(first[b]) + i for i in range(kept[b])]
        assert (sv.spec_cache_resize(k, v, *book, advance=d(kept))["status"] == 0).all()
        if rng.random() < 0.4:
            src, dst = rng.permutation(B)[:2]
            assert sv.spec_cache_fork(d([src]), d([dst]), *book, P)["status"].tolist() == [0]
            tokens[dst] = list(tokens[src])
        assert length.tolist() == [len(t) for t in tokens]
        kc, vc, tc = k.cpu().numpy(), v.cpu().numpy(), table.cpu().numpy()
        for b in range(B):
            pos = np.arange(len(tokens[b]))
            page = tc[b][pos // P]
            want = np.array(tokens[b], np.float32)
            for layer in range(2):
                got = kc[layer, page, 0, pos % P]
                assert (got == (want + np.float32(0.25 * layer))[:, None]).all(), (step, b, layer)
                assert (vc[layer, page, 0, pos % P] == -got).all()
        count = np.zeros(pages, np.int64)
        for b in range(B):
            np.add.at(count, tc[b][:int(held[b])], 1)
        assert (count == refs.cpu().numpy()).all()
    assert waited > 0 and (passed > 0) == longer
