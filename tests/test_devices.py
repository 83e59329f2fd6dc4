"""Tensors of another device than the current one are refused where a call takes its stream (CPU only: the
devices are fakes)."""

import pytest

torch = pytest.importorskip("torch")


class OnDevice:
    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


@pytest.mark.parametrize("name", ["_stream_of", "_stream"])
def test_another_device_is_refused(monkeypatch, name):
    from bit_quantized_moe_quantize_gb300 import _lib
    monkeypatch.setattr(_lib, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        getattr(_lib, name)(1 if name == "_stream_of" else OnDevice(1))
