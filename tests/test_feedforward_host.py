"""Host side of the feed-forward binding, without a GPU."""
import pytest

from mxfp4_w4a4_quantized_amd import feedforward as ff


def test_default_stream_of_another_gpu_is_refused(monkeypatch):
    """A GPU's default stream has the handle 0, which a launch takes for the
    current GPU's: the kernels would run there, on the other GPU's addresses."""
    monkeypatch.setattr(ff, "_current_device", lambda: 0)
    monkeypatch.setattr(ff, "_raw_stream", lambda dev: 0)
    assert ff._stream(0) == 0
    with pytest.raises(ValueError, match="GPU 1"):
        ff._stream(1)
    monkeypatch.setattr(ff, "_raw_stream", lambda dev: 1000 + dev)   # a stream of its own
    assert ff._stream(0) == 1000 and ff._stream(1) == 1001
