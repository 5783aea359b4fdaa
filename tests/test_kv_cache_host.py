"""Host side of the KV-cache calls' Python binding (no GPU needed)."""

import pytest


@pytest.fixture(scope="module")
def lib():
    from long_context_attention_compress_b200 import build as b
    b.build()
    from long_context_attention_compress_b200 import _lib
    return _lib


def test_current_device_without_the_short_cut(lib, monkeypatch):
    """A torch without the private call for the device's number, and one with it: the public call's answer."""
    monkeypatch.setattr(lib.torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(lib.torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(lib, "_raw_device", lambda: 5)
    assert lib._current_device() == 5
    monkeypatch.setattr(lib, "_raw_device", None)
    assert lib._current_device() == 3
    monkeypatch.delattr(lib.torch._C, "_cuda_getDevice", raising=False)
    assert lib._current_device() == 3
