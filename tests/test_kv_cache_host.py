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


def test_empty_batch_with_a_selection(lib):
    """No queries, so no index array (an empty tensor has no address), but its width is given: nothing to do."""
    import ctypes
    from types import SimpleNamespace
    cfg = lib.make_cfg(SimpleNamespace(c=512, m=4, m_hca=128, topk=1024, n_idx_heads=64, d_idx=128, n_heads=64, n_win=128,
                                       scale=512 ** -0.5, rope_dims=64, rope_base=1e4, norm_eps=1e-6))
    d = lib.KvCacheDesc()
    for k, v in dict(form=2, c=512, rope_dims=64, codes=0x10000, scales=0x10000, rope=0x10000, ld_codes=224, ld_scales=16,
                     ld_rope=64, n_rows=512, n_req=4, seq_rows=128).items():
        setattr(d, k, v)

    def call(Tq, n_idx):
        return lib._mqa_fp4(None, ctypes.byref(d), 128, None, n_idx, 4, None, 0, 0, None, None, Tq, ctypes.byref(cfg), None, 0,
                            None, None, 0, None)
    assert call(0, 1024) == 0 and call(0, 0) == 0
    assert call(4, 1024) == -1 and call(0, -1) == -1
