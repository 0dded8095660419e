"""What the cache calls' binding checks before it hands pointers to the library (CPU only)."""

from types import SimpleNamespace

import pytest

import speculative_decoding_block_verify_gb300 as sv

torch = pytest.importorskip("torch")


def test_launches_go_to_the_current_device(monkeypatch):
    fake = SimpleNamespace(_C=SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda d: 100 + d))
    monkeypatch.setattr(sv, "_T", fake)
    monkeypatch.setattr(sv, "_ONE_DEVICE", False, raising=False)
    side = SimpleNamespace(device_index=0, cuda_stream=7)
    assert sv._raw_stream(None, 0) == 100 and sv._raw_stream(side, 0) == 7
    with pytest.raises(ValueError, match="current device is cuda:0"):
        sv._raw_stream(None, 1)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        sv._raw_stream(SimpleNamespace(device_index=1, cuda_stream=7), 1)
    with pytest.raises(ValueError, match="stream on cuda:1"):
        sv._raw_stream(SimpleNamespace(device_index=1, cuda_stream=7), 0)
    # with a single device there is nothing to compare
    monkeypatch.setattr(sv, "_ONE_DEVICE", True)
    assert sv._raw_stream(None, 0) == 100 and sv._raw_stream(side, 0) == 7


def test_a_workspace_has_to_be_on_the_device():
    ws = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(TypeError, match="workspace"):
        sv._space(ws, 0)
    assert sv._space(ws, -1) == (ws.data_ptr(), 512)
    assert sv._space(ws.view(torch.int32), -1)[1] == 512
    with pytest.raises(TypeError, match="workspace"):
        sv._space(ws[::2], -1)
