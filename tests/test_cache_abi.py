"""The cache calls' host side: argument structs as the C compiler lays them out, and errors that are answered before
any launch (CPU only)."""

import ctypes

import pytest

import speculative_decoding_block_verify_gb300 as sv
from speculative_decoding_block_verify_gb300 import build as svbuild


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


P = 4096   # a pointer that is never followed: the checks come first


def attention(**kw):
    a = dict(B=2, kmax=5, Hq=8, Hkv=2, D=64, page=16, pages=100, width=10, dtype=1, window=0, sinks=0, scale=0.125, cu=P,
             length=P, table=P, q=P, stride=8 * 64, rows=12, k=P, v=P, out=P, status=P, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return sv._ATTENTION.pack(*a.values())


def append(**kw):
    a = dict(B=2, kmax=5, Hkv=2, D=64, page=16, pages=100, width=10, dtype=1, cu=P, length=P, table=P, k=P, v=P, ks=128, vs=128,
             rows=12, kp=P, vp=P, status=P)
    a.update(kw)
    return sv._APPEND.pack(*a.values())


def resize(**kw):
    a = dict(B=2, page=16, pages=100, width=10, layers=2, bytes=4096, advance=P, room=P, table=P, held=P, length=P, refs=P, k=P,
             v=P, status=P, ws=P, ws_bytes=1 << 20)
    a.update(kw)
    return sv._RESIZE.pack(*a.values())


def test_struct_sizes():
    assert (sv._ATTENTION.size, sv._APPEND.size, sv._RESIZE.size) == (144, 120, 120)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), -2), (dict(B=-1), -3), (dict(B=65536), -3), (dict(kmax=33), -3), (dict(kmax=-1), -3), (dict(Hq=9), -3),
    (dict(Hkv=0), -3), (dict(Hq=129, Hkv=1, stride=129 * 64), -3), (dict(D=60), -3), (dict(D=264), -3), (dict(page=24), -3),
    (dict(page=512), -3), (dict(page=4), -3), (dict(pages=0), -3), (dict(width=0), -3), (dict(width=1 << 28), -3),
    (dict(window=-1), -3), (dict(sinks=-1), -3), (dict(stride=511), -3), (dict(rows=-1), -3), (dict(cu=0, rows=11), -3),
    (dict(length=0), -1), (dict(table=0), -1), (dict(q=0), -1), (dict(k=0), -1), (dict(out=0), -1), (dict(status=0), -1),
    (dict(k=P + 8), -1), (dict(v=P + 2), -1), (dict(out=P + 8), -1), (dict(scale=float("nan")), -1)])
def test_attention_errors(L, change, code):
    assert L.spec_paged_attention(attention(**change), None) == code
    assert L.spec_last_error() != b""


def test_append_errors(L):
    for change, code in [(dict(dtype=-1), -2), (dict(B=-1), -3), (dict(kmax=33), -3), (dict(D=12), -3), (dict(Hkv=0), -3), (dict(page=20), -3),
                         (dict(ks=127), -3), (dict(vs=0), -3), (dict(rows=-1), -3), (dict(cu=0, rows=11), -3), (dict(k=0), -1), (dict(v=0), -1),
                         (dict(kp=0), -1), (dict(vp=P + 8), -1), (dict(status=0), -1), (dict(table=0), -1)]:
        assert L.spec_cache_append(append(**change), None) == code, change
    assert L.spec_cache_append(append(B=0), None) == 0


def test_resize_errors(L):
    for change, code in [(dict(B=-1), -3), (dict(B=65536), -3), (dict(page=12), -3), (dict(pages=0), -3), (dict(width=0), -3), (dict(layers=0), -3),
                         (dict(bytes=8), -3), (dict(bytes=24), -3), (dict(table=0), -1), (dict(held=0), -1), (dict(refs=0), -1), (dict(k=0), -1),
                         (dict(v=P + 4), -1), (dict(status=0), -1), (dict(ws=0), -6), (dict(ws=P + 8), -6), (dict(ws_bytes=100), -6)]:
        assert L.spec_cache_resize(resize(**change), None) == code, change
    assert L.spec_cache_resize(resize(B=0), None) == 0
    assert L.spec_cache_resize_workspace_bytes(0, 10) == 0 and L.spec_cache_resize_workspace_bytes(4, 0) == 0
    # a header, the copies (8 bytes) and two words a stream, and a word a page
    assert L.spec_cache_resize_workspace_bytes(64, 1000) == 256 + 4 * 256 + 4000


def test_fork_errors(L):
    vp = ctypes.c_void_p
    ok = [P, P, 2, 4, 16, 100, 10, P, P, P, P, P]
    for at, value, code in [(2, -1, -3), (3, -1, -3), (3, 65536, -3), (4, 17, -3), (5, 0, -3), (6, 0, -3), (0, 0, -1), (1, 0, -1), (7, 0, -1),
                            (8, 0, -1), (9, 0, -1), (10, 0, -1), (11, 0, -1)]:
        a = list(ok)
        a[at] = value
        assert L.spec_cache_fork(*a, vp(0)) == code, (at, value)
    assert L.spec_cache_fork(*(ok[:2] + [0] + ok[3:]), vp(0)) == 0


def test_null_arguments_and_empty_batches(L):
    assert L.spec_paged_attention(None, None) == -1
    assert L.spec_cache_append(None, None) == -1
    assert L.spec_cache_resize(None, None) == -1
    assert L.spec_paged_attention_workspace_bytes(None) == 0
    assert L.spec_paged_attention_workspace_bytes(attention(D=3)) == 0
    assert L.spec_paged_attention(attention(B=0), None) == 0
    assert L.spec_last_error() == b""
