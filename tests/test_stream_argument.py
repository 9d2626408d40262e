"""Which stream a call goes to."""
import types

import pytest

import sample_gradient_clipping_amd as dp


def test_the_current_stream_with_and_without_torchs_raw_accessor(monkeypatch):
    torch = pytest.importorskip("torch")
    t = types.SimpleNamespace(device=torch.device("cuda", 3))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=200 + device.index))
    assert dp._stream(t, None) == 103
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert dp._stream(t, None) == 203
    assert dp._stream(t, types.SimpleNamespace(cuda_stream=7)) == 7 and dp._stream(t, 9) == 9
