"""Caches that kv_cache_append fills, read by the framework's other calls: the FP4 indexer's keys, and the newest entry that
the decode layer call appends to an FP4 cache."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import Cache
from long_context_attention_compress_b200 import workloads as wl
from parity_util import to64

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("norm", [False, True])
def test_appended_keys_are_the_indexers(norm):
    """Indexer keys of three requests appended in two ragged chunks and then one a request, into the flat layout that
    csa_indexer_topk_fp4 reads: the arrays and the selection that mxfp4_quantize's keys give."""
    import long_context_attention_compress_b200 as hca
    s = wl.PRO
    cfg = hca.make_cfg(s)
    B, N = 3, 5000
    g = torch.Generator().manual_seed(6)
    K = torch.randn(B, N, 128, generator=g).bfloat16().cuda()
    gamma = (torch.rand(128, generator=g) + 0.5).cuda() if norm else None
    codes = torch.full((B, N, 64), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((B, N, 4), 0xFF, dtype=torch.uint8, device="cuda")
    cache = hca.KvCache("fp4", 128, 0, codes, scales)
    for at, counts in (([0, 0, 0], [4000, 17, 4999]), ([4000, 17, 4999], [999, 4983, 0])):
        x = torch.cat([K[b, a:a + n] for b, (a, n) in enumerate(zip(at, counts))])
        hca.kv_cache_append(x, cache, _i32(at), row_start=_i32(np.concatenate([[0], np.cumsum(counts)])), gamma=gamma)
    hca.kv_cache_append(K[:, N - 1].contiguous(), cache, _i32([N - 1, -1, N - 1]), gamma=gamma)
    keys = K.reshape(B * N, 128)
    if norm:
        keys = torch.tensor(oracle.round_bf16(oracle.rms_norm(to64(keys), gamma.double().cpu().numpy(), 1e-6))).bfloat16().cuda()
    want_c, want_s = (t.reshape(B, N, -1) for t in hca.mxfp4_quantize(keys))
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    q = torch.randn(B, s.n_idx_heads, s.d_idx, generator=g).bfloat16().cuda()
    w = torch.randn(B, s.n_idx_heads, generator=g).cuda()
    pos = _i32([s.m * N - 1, s.m * 4500 + 1, s.m * N - 1])
    assert torch.equal(hca.csa_indexer_topk_fp4(q, w, codes, scales, pos, cfg),
                       hca.csa_indexer_topk_fp4(q, w, want_c, want_s, pos, cfg))


@pytest.mark.parametrize("rpb", [0, 1])
@pytest.mark.parametrize("norm", [False, True])
def test_newest_entry_of_the_layer_call(rpb, norm):
    """The appended entry's scales are those of the exact entry's stored form and its codes are equal or neighbours, which
    they are only next to a rounding border: the compressor's f32 entry is within 2^-18 of its group's largest, so that at
    most one code in a hundred can turn (one in thirty after the rounding to bf16, whose step is 2^-8)."""
    import long_context_attention_compress_b200 as hca
    s = wl.PRO
    cfg = hca.make_cfg(s)
    B, ctx = 8, 128 * 40
    d = wl.hca_decode_inputs(s, B, ctx, seed=71, with_block=True)
    Nh = d["E_h"].shape[1]
    k = Cache("fp4", s.c, 64, B, Nh, rpb=rpb, seed=5, fill=0)
    gh = {n: v.cuda() for n, v in d.items() if n != "E_h"} | {"N": Nh}
    w = wl.norm_weights(s, seed=4)
    out = torch.empty((B, s.n_heads, s.c), dtype=torch.bfloat16, device="cuda")
    args, keep = hca.make_decode_args(B, gh["q_pos"], hca=gh, hca_out=out, hca_kv4=k.handle,
                                      **({"hca_norm": w.cuda()} if norm else {}))
    ws = torch.empty((hca.hybrid_attn_decode_workspace(cfg, args),), dtype=torch.uint8, device="cuda")
    hca.hybrid_attn_decode(cfg, args, ws=ws)
    new = np.concatenate([oracle.hca_compress(to64(d["block_cand"][b]), to64(d["block_logits"][b]),
                                              d["bias_hca"].double().numpy(), s.m_hca).reshape(1, -1) for b in range(B)])
    if norm:
        new = oracle.round_bf16(oracle.rope(oracle.rms_norm(new, w[1].double().numpy(), s.norm_eps),
                                            oracle.entry_position(Nh - 1, s.m_hca), 64, 10000.0))
    codes, scales = oracle.mxfp4_quantize(new[:, :448])
    rows = [k.row(b, Nh - 1) for b in range(B)]
    have = {n: v[rows] for n, v in k.bytes().items()}
    got = oracle.mxfp4_unpack(have["codes"])
    np.testing.assert_array_equal(have["scales"][:, :14], scales)
    value = lambda c: np.where(c & 8, -(c & 7).astype(int), c & 7)  # noqa: E731  (codes of one sign ascend)
    step = np.abs(value(got) - value(codes))
    assert step.max() <= 1 and np.mean(step > 0) <= (1 / 30 if norm else 1 / 100), (step.max(), np.mean(step > 0))
    rope = to64(torch.tensor(have["rope"]).view(torch.bfloat16))
    assert np.all(np.abs(rope - new[:, 448:]) <= 2.0 ** -7 * np.abs(new[:, 448:]) + 1e-6)


def test_fp4_hca_cache_runs_beside_the_indexer():
    """The hybrid decode step of 8 requests at 1M tokens with an FP4 HCA cache: its attention overlaps the indexer as the
    bf16 one does (one after the other the step took 1.63 times as long; a fifth is allowed for noise)."""
    import long_context_attention_compress_b200 as hca
    s = wl.PRO
    cfg = hca.make_cfg(s)
    B, ctx = 8, 1 << 20
    d = wl.hybrid_decode_inputs(s, B, ctx, seed=1, device="cuda")
    Nh = d["hca"]["E_h"].shape[1]
    t = {"codes": torch.empty(B, Nh, 224, dtype=torch.uint8, device="cuda"),
         "scales": torch.empty(B, Nh, 16, dtype=torch.uint8, device="cuda"),
         "rope": torch.empty(B, Nh, 64, dtype=torch.bfloat16, device="cuda")}
    k = hca.KvCache("fp4", s.c, 64, **t)
    hca.kv_cache_append(d["hca"]["E_h"].reshape(B * Nh, s.c), k, _i32([0] * B), row_start=_i32(np.arange(B + 1) * Nh))
    idx = torch.empty((B, s.topk), dtype=torch.int32, device="cuda")
    oc = torch.empty((B, s.n_heads, s.c), dtype=torch.bfloat16, device="cuda")
    oh = torch.empty_like(oc)
    calls = []
    for gh, kw in ((d["hca"], {}), ({n: v for n, v in d["hca"].items() if n != "E_h"} | {"N": Nh}, {"hca_kv4": k})):
        args, keep = hca.make_decode_args(B, d["csa"]["q_pos"], csa=d["csa"], hca=gh, csa_topk_idx=idx, csa_out=oc,
                                          hca_out=oh, **kw)
        ws = torch.empty((hca.hybrid_attn_decode_workspace(cfg, args),), dtype=torch.uint8, device="cuda")
        calls.append((args, keep, ws))
    times = ([], [])
    for i in range(60):
        args, _, ws = calls[i % 2]
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        hca.hybrid_attn_decode(cfg, args, ws=ws)
        b.record()
        torch.cuda.synchronize()
        times[i % 2].append(a.elapsed_time(b))
    bf16, fp4 = (float(np.median(v[5:])) for v in times)
    assert fp4 <= 1.2 * bf16, (bf16, fp4)
