"""Host-side checks of kv_cache_append, kv_cache_gather and sparse_mqa_attend_fp4: every call here is refused, or has
nothing to do, before anything is launched (no GPU needed)."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from long_context_attention_compress_b200 import build as b
    b.build()
    from long_context_attention_compress_b200 import _lib
    return _lib


FAKE = 0x10000  # aligned, never dereferenced


def desc(lib, form=2, **kw):
    d = lib.KvCacheDesc()
    n = 448
    vals = dict(form=form, c=512, rope_dims=64, codes=FAKE, scales=FAKE, rope=FAKE,
                ld_codes={0: 512, 1: n, 2: n // 2}.get(form, 512), ld_scales={1: 7, 2: 16}.get(form, 0), ld_rope=64,
                n_rows=4 * 128, n_req=4, ring=0, seq_rows=128, block_table=None, bt_stride=0, rows_per_block=0)
    vals.update(kw)
    for k, v in vals.items():
        setattr(d, k, v)
    return d


def append(lib, d, **kw):
    a = dict(x=FAKE, f32=1, ld=512, n=4, start=None, first=FAKE, B=4, rate=4, gamma=FAKE, eps=1e-6, rot=1, base=1e4)
    a.update(kw)
    return lib._kv_append(a["x"], a["f32"], a["ld"], a["n"], a["start"], a["first"], a["B"], a["rate"], a["gamma"],
                          a["eps"], a["rot"], a["base"], ctypes.byref(d) if d else None, None)


def gather(lib, d, **kw):
    a = dict(B=4, n=8, idx=None, first=None, out=FAKE, ld=512, seq=4096)
    a.update(kw)
    return lib._kv_gather(ctypes.byref(d) if d else None, a["B"], a["n"], a["idx"], a["first"], a["out"], a["ld"],
                          a["seq"], None)


@pytest.mark.parametrize("form", [0, 1, 2])
def test_cache_descriptor_refusals(lib, form):
    for call in (append, gather):
        for st, kw in [(-1, dict(form=3)), (-1, dict(form=-1)), (-1, dict(c=0)), (-1, dict(rope_dims=-8)),
                       (-1, dict(rope_dims=520)), (-2, dict(c=516)), (-2, dict(c=520, rope_dims=8)), (-2, dict(rope_dims=60)),
                       (-2, dict(c=512, rope_dims=264)), (-1, dict(codes=None)), (-1, dict(codes=FAKE + 8)),
                       (-1, dict(n_rows=-1)), (-1, dict(n_req=-1)), (-1, dict(seq_rows=0)), (-1, dict(seq_rows=129)),
                       (-1, dict(block_table=FAKE, bt_stride=0, rows_per_block=8)),
                       (-1, dict(block_table=FAKE + 2, bt_stride=4, rows_per_block=8)),
                       (-1, dict(block_table=FAKE, bt_stride=4, rows_per_block=0)),
                       (-2, dict(block_table=FAKE, bt_stride=4, rows_per_block=8, ring=1))]:
            assert call(lib, desc(lib, **dict(dict(form=form), **kw))) == st, (call.__name__, kw, lib.last_error())
            assert lib.last_error()
        assert call(lib, None) == -1
        if form == 0:
            assert call(lib, desc(lib, form, ld_codes=504)) == -1 and call(lib, desc(lib, form, ld_codes=516)) == -1
        else:
            assert call(lib, desc(lib, form, rope_dims=56)) == -2     # 456 channels: no whole groups
            assert call(lib, desc(lib, form, rope_dims=0, c=0)) == -1
            assert call(lib, desc(lib, form, ld_codes=200 if form == 2 else 432)) == -1
            assert call(lib, desc(lib, form, ld_codes=232 if form == 2 else 456)) == -1
            assert call(lib, desc(lib, form, ld_scales=13 if form == 2 else 6)) == -1
            assert call(lib, desc(lib, form, scales=None)) == -1
            assert call(lib, desc(lib, form, rope=None)) == -1 and call(lib, desc(lib, form, rope=FAKE + 8)) == -1
            assert call(lib, desc(lib, form, ld_rope=56)) == -1 and call(lib, desc(lib, form, ld_rope=68)) == -1
    assert append(lib, desc(lib, 1, scales=FAKE + 2)) == -1


def test_append_refusals(lib):
    d = desc(lib)
    assert append(lib, d, n=0, B=0) == 0 and append(lib, d, n=0, start=FAKE) == 0
    assert append(lib, d, n=5) == -1 and "row_start" in lib.last_error()
    assert append(lib, d, n=5, B=5) == -1                       # the cache has 4 requests
    assert append(lib, d, n=-1) == -1 and append(lib, d, B=-1, n=-1) == -1
    assert append(lib, d, n=(1 << 30) + 1, start=FAKE) == -1
    assert append(lib, d, rate=0) == -1
    assert append(lib, d, ld=504) == -1 and append(lib, d, ld=514) == -1 and append(lib, d, f32=0, ld=516) == -1
    assert append(lib, d, x=None) == -1 and append(lib, d, x=FAKE + 8) == -1
    assert append(lib, d, first=None) == -1 and append(lib, d, first=FAKE + 1) == -1
    assert append(lib, d, start=FAKE + 2) == -1
    assert append(lib, d, gamma=FAKE + 4) == -1 and append(lib, d, eps=-1.0) == -1
    assert append(lib, d, base=0.0) == -1


def test_gather_refusals(lib):
    d = desc(lib)
    assert gather(lib, d, B=0) == 0 and gather(lib, d, n=0) == 0
    assert gather(lib, d, B=5) == -1 and gather(lib, d, B=-1) == -1 and gather(lib, d, n=-1) == -1
    assert gather(lib, d, n=(1 << 29) + 1) == -1
    assert gather(lib, d, idx=FAKE, first=FAKE) == -1 and "both" in lib.last_error()
    assert gather(lib, d, out=None) == -1 and gather(lib, d, out=FAKE + 8) == -1
    assert gather(lib, d, ld=504) == -1 and gather(lib, d, ld=516) == -1 and gather(lib, d, seq=-8) == -1
    assert gather(lib, d, idx=FAKE + 2) == -1 and gather(lib, d, first=FAKE + 1) == -1


def test_attend_refusals(lib):
    from types import SimpleNamespace
    shape = dict(c=512, m=4, m_hca=128, topk=1024, n_idx_heads=64, d_idx=128, n_heads=64, n_win=128, scale=512 ** -0.5,
                 rope_dims=64, rope_base=1e4, norm_eps=1e-6)
    cfg = lambda **kw: lib.make_cfg(SimpleNamespace(**dict(shape, **kw)))  # noqa: E731
    need = lib.sparse_mqa_attend_fp4_workspace(cfg(), 4, 8192, 0)
    assert 0 < need < lib.SIZE_MAX and need % 256 == 0

    def call(**kw):
        a = dict(q=FAKE, d=desc(lib), N=8192, idx=None, k=0, rate=4, win=FAKE, ws_=128 * 512, W=128, pos=FAKE, req=None, Tq=4,
                 cfg=cfg(), sink=None, rot=0, out=FAKE, ws=FAKE, nb=1 << 30)
        a.update(kw)
        return lib._mqa_fp4(a["q"], ctypes.byref(a["d"]) if a["d"] else None, a["N"], a["idx"], a["k"], a["rate"], a["win"],
                            a["ws_"], a["W"], a["pos"], a["req"], a["Tq"], ctypes.byref(a["cfg"]), a["sink"], a["rot"],
                            a["out"], a["ws"], a["nb"], None)

    assert call(Tq=0, nb=0, ws=None) == 0
    assert call(nb=need - 1) == -3 and "workspace" in lib.last_error()
    for bad in (dict(c=0), dict(n_heads=0), dict(n_win=0), dict(scale=0.0), dict(c=256)):
        assert call(cfg=cfg(**bad)) == -1, bad
    for bad in (dict(n_heads=129), dict(c=520), dict(c=1024)):
        assert call(cfg=cfg(**bad)) == -2, bad
        assert lib.sparse_mqa_attend_fp4_workspace(cfg(**bad), 4, 100, 0) == lib.SIZE_MAX
    assert lib.sparse_mqa_attend_fp4_workspace(cfg(), -1, 100, 0) == lib.SIZE_MAX
    assert lib.sparse_mqa_attend_fp4_workspace(cfg(), 4, 100, 4097) == lib.SIZE_MAX
    assert lib.sparse_mqa_attend_fp4_workspace(cfg(), 0, 100, 0) == 0
    assert call(d=None) == -1
    assert call(d=desc(lib, 0)) == -2 and call(d=desc(lib, 1)) == -2 and call(d=desc(lib, ring=1)) == -2
    assert call(d=desc(lib, scales=FAKE + 8)) == -1 and call(d=desc(lib, ld_scales=14)) == -1
    assert call(Tq=-1) == -1 and call(N=-1) == -1 and call(rate=0) == -1
    assert call(N=(1 << 30) + 1) == -1 and call(Tq=(1 << 20) + 1, req=FAKE) == -1
    assert call(cfg=cfg(n_win=(1 << 20) + 1), W=(1 << 20) + 1, ws_=((1 << 20) + 1) * 512) == -2
    assert lib.sparse_mqa_attend_fp4_workspace(cfg(), 4, (1 << 30) + 1, 0) == lib.SIZE_MAX
    assert call(idx=FAKE) == -1 and call(k=5) == -1 and call(idx=FAKE, k=4097) == -1
    assert call(Tq=5) == -1 and "q_req" in lib.last_error()
    assert call(W=127) == -1 and call(ws_=128 * 512 + 4) == -1 and call(ws_=128 * 512 - 8) == -1
    assert call(rot=1, cfg=cfg(rope_dims=0)) == -1 and call(rot=1, cfg=cfg(rope_dims=12)) == -1
    assert call(rot=1, cfg=cfg(rope_base=0.0)) == -1
    assert call(q=None) == -1 and call(q=FAKE + 8) == -1 and call(out=None) == -1 and call(win=FAKE + 8) == -1
    assert call(pos=None) == -1 and call(pos=FAKE + 2) == -1 and call(req=FAKE + 1) == -1 and call(sink=FAKE + 2) == -1
    assert call(idx=FAKE + 2, k=4) == -1
    assert call(ws=None) == -1 and call(ws=FAKE + 128) == -1


def test_layer_decode_refusals(lib):
    """csa_kv4 / hca_kv4 of hybrid_attn_decode: each bad cache is refused by the call, and those that change the plan by
    the workspace query too."""
    from types import SimpleNamespace
    cfg = lib.make_cfg(SimpleNamespace(c=512, m=4, m_hca=128, topk=64, n_idx_heads=64, d_idx=128, n_heads=64, n_win=128,
                                       scale=512 ** -0.5, rope_dims=64, rope_base=1e4, norm_eps=1e-6))
    kv8 = lib.KvFp8()

    def call(layer, d, B=2, query=False, **kw):
        a = lib.DecodeArgs()
        a.B, a.q_pos = B, FAKE
        names = dict(q=FAKE, out=FAKE, N=8192, win=FAKE, win_stride=128 * 512)
        if layer == "csa":
            names.update(q_idx=FAKE, w_idx=FAKE, k_idx=FAKE, k_stride=128 * 128, topk_idx=FAKE)
        names.update(kw)
        for k, v in names.items():
            setattr(a, f"{layer}_{k}", v)
        setattr(a, f"{layer}_kv4", ctypes.addressof(d))
        if query:
            return lib.hybrid_attn_decode_workspace(cfg, a)
        return lib._decode(ctypes.byref(cfg), ctypes.byref(a), None, 0, None)

    for layer in ("csa", "hca"):
        cache = lambda **kw: desc(lib, **dict(dict(n_rows=4 * 8192, seq_rows=8192), **kw))  # noqa: E731
        assert 0 < call(layer, cache(), query=True) < lib.SIZE_MAX
        assert call(layer, cache()) == -3 and "workspace" in lib.last_error()    # everything else is in order
        assert call(layer, cache(block_table=FAKE, bt_stride=1024, rows_per_block=8)) == -3
        for st, kw in [(-2, dict(form=0)), (-2, dict(form=1)), (-2, dict(ring=1)), (-1, dict(c=256, rope_dims=64, ld_codes=96)),
                       (-1, dict(n_req=1, n_rows=8192)), (-1, dict(scales=FAKE + 8)), (-1, dict(ld_scales=24)),
                       (-2, dict(n_rows=1 << 31)), (-1, dict(codes=None))]:
            d = cache(**kw)
            assert call(layer, d) == st, (layer, kw, lib.last_error())
            assert call(layer, d, query=True) == lib.SIZE_MAX, (layer, kw)
        assert call(layer, cache(), N=8193) == -1 and "room" in lib.last_error()
        assert call(layer, cache(block_table=FAKE, bt_stride=1023, rows_per_block=8)) == -1
        assert call(layer, cache(), win_stride=127 * 512) == -1
        assert call(layer, cache(), kv8=ctypes.addressof(kv8)) == -1 and "both" in lib.last_error()
        assert call(layer, cache(rope_dims=0, ld_codes=256), norm=FAKE) == -1 and "rope_dims" in lib.last_error()
        assert call(layer, cache(rope_dims=0, ld_codes=256)) == -3


def test_fault_injection(lib, monkeypatch):
    monkeypatch.setenv("HCA_INJECT_FAULT", "all")
    assert append(lib, desc(lib)) == -6 and gather(lib, desc(lib)) == -6


def test_handle_refuses_wrong_tensors(lib):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):
        lib.KvCache("fp4", 512, 64, u8(2, 8, 224), u8(2, 8, 16), torch.zeros(2, 8, 64, dtype=torch.bfloat16))  # CPU
    with pytest.raises(ValueError):
        lib.KvCache("int4", 512, 64, u8(2, 8, 224))
    with pytest.raises(TypeError):
        lib.KvCache("fp4", 512, 64, None)
