"""FP4 caches in use on the GPU: the decode layer call over them (csa_kv4 / hca_kv4), and a prompt and decode steps made
of the single calls (append, read back, attend).  Outputs are held to the bounds of test_gpu_mqa_fp4 against float64
attention over the rows that the caches' bytes stand for; the bytes that the calls append are checked on their own."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import Cache, fill_rows, values
from long_context_attention_compress_b200 import workloads as wl
from parity_util import check_topk_row, to64
from test_gpu_mqa_fp4 import check_query

pytestmark = pytest.mark.gpu


def _cache_of(E, rpb, seed):
    """An FP4 cache holding rows E [B, N, c] (float64)."""
    B, N, c = E.shape
    k = Cache("fp4", c, 64, B, N, rpb=rpb, seed=seed, fill=0xFF)
    fill_rows(k, [k.row(b, e) for b in range(B) for e in range(N)], E.reshape(B * N, c))
    return k


def _rows(k, b, entries):
    ref = values("fp4", k.bytes(), {n: k.width(n) for n in k.t}, 64)
    return ref[[k.row(b, int(e)) for e in entries]]


@pytest.mark.parametrize("case", ["flat", "paged", "norm", "fp4_keys", "csa_only", "hca_only"])
def test_layer_decode_from_fp4_caches(case):
    import long_context_attention_compress_b200 as hca
    s = wl.PRO
    cfg = hca.make_cfg(s)
    B, ctx = 2, 4 * 5120
    t = ctx - 1
    csa = wl.csa_decode_inputs(s, B, ctx, seed=61)
    hcd = wl.hca_decode_inputs(s, B, ctx, seed=62, with_block=True)
    rpb_c, rpb_h = (32, 1) if case in ("paged", "norm") else (0, 0)
    kc = _cache_of(to64(csa["E"]), rpb_c, 1)
    kh = _cache_of(to64(hcd["E_h"]), rpb_h, 2)
    N, Nh = csa["E"].shape[1], hcd["E_h"].shape[1]
    gc = {k: v.cuda() for k, v in csa.items() if k != "E"} | {"N": N}
    gh = {k: v.cuda() for k, v in hcd.items() if k != "E_h"} | {"N": Nh}
    sink = torch.randn(2, s.n_heads, generator=torch.Generator().manual_seed(3))
    kw = {"csa_sink": sink[0].cuda(), "hca_sink": sink[1].cuda()} if case != "norm" else {}
    nrm = {}
    if case == "norm":
        kw = {"csa_norm": wl.norm_weights(s, seed=3).cuda(), "hca_norm": wl.norm_weights(s, seed=4).cuda()}
        nrm = {k: v.double().cpu().numpy() for k, v in kw.items()}
    if case == "fp4_keys":
        kw["csa_k4"] = tuple(x.reshape(B, N, -1) for x in hca.mxfp4_quantize(csa["K_I"].reshape(B * N, -1).cuda()))
    idx = torch.empty((B, s.topk), dtype=torch.int32, device="cuda")
    oc = torch.empty((B, s.n_heads, s.c), dtype=torch.bfloat16, device="cuda")
    oh = torch.empty_like(oc)
    args, keep = hca.make_decode_args(B, gc["q_pos"], csa=gc if case != "hca_only" else None,
                                      hca=gh if case != "csa_only" else None, csa_topk_idx=idx, csa_out=oc, hca_out=oh,
                                      csa_kv4=kc.handle, hca_kv4=kh.handle, **kw)
    need = hca.hybrid_attn_decode_workspace(cfg, args)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    before = kh.bytes()
    for _ in range(2):  # the second call finds the entry there, and gives the same bits
        hca.hybrid_attn_decode(cfg, args, ws=ws)
        got = (oc.clone(), oh.clone())
    torch.cuda.synchronize()
    assert hca.lib.hca_check_device() == 0, hca.last_error()
    assert torch.equal(got[0].view(torch.int16), oc.view(torch.int16)) and torch.equal(got[1].view(torch.int16),
                                                                                       oh.view(torch.int16))

    def prep(q, win, norm, b):
        """Queries and window rows as they are attended."""
        q, win = to64(q[b]), to64(win[b])
        if norm is None:
            return q, win, None
        nr = lambda x, g, pos: oracle.round_bf16(oracle.rope(oracle.rms_norm(x, g, s.norm_eps), pos, 64, 10000.0))  # noqa: E731
        return nr(q, norm[0], t), nr(win, norm[1], np.arange(t - s.n_win + 1, t + 1)), t

    for b in range(B):
        if case != "hca_only":
            if case != "fp4_keys":
                sc = oracle.indexer_scores(to64(csa["q_idx"][b]), csa["w_idx"][b].double().numpy(), to64(csa["K_I"][b]))
                check_topk_row(idx[b].cpu().numpy(), oracle.topk_select(sc, s.topk), sc, s.topk, N)
            q, win, rot = prep(csa["q"], csa["win"], nrm.get("csa_norm"), b)
            check_query(to64(oc[b]), q, np.concatenate([_rows(kc, b, idx[b].cpu().numpy()), win]), s.scale,
                        sink[0].double().numpy() if "csa_sink" in kw else None, rot, what=f"csa {b}")
        if case != "csa_only":
            # the newest entry: within one E2M1 step of the exact one, its block's exponent within one
            new = oracle.hca_compress(to64(hcd["block_cand"][b]), to64(hcd["block_logits"][b]),
                                      hcd["bias_hca"].double().numpy(), s.m_hca)
            if nrm:
                new = oracle.round_bf16(oracle.rope(oracle.rms_norm(new, nrm["hca_norm"][1], s.norm_eps),
                                                    oracle.entry_position(Nh - 1, s.m_hca), 64, 10000.0))
            have = _rows(kh, b, [Nh - 1])
            assert np.all(np.abs(have - new) <= 0.5 * np.abs(new) + 2.0 ** -3 * np.abs(new).max())
            assert np.all(np.abs(have[:, 448:] - new[:, 448:]) <= 2.0 ** -7 * np.abs(new[:, 448:]) + 1e-6)
            q, win, rot = prep(hcd["q"], hcd["win"], nrm.get("hca_norm"), b)
            check_query(to64(oh[b]), q, np.concatenate([_rows(kh, b, range(Nh)), win]), s.scale,
                        sink[1].double().numpy() if "hca_sink" in kw else None, rot, what=f"hca {b}")
    if case != "csa_only":
        new_rows = [kh.row(b, Nh - 1) for b in range(B)]
        for name, v in kh.bytes().items():
            keep_rows = np.ones(v.shape[0], bool)
            keep_rows[new_rows] = False
            np.testing.assert_array_equal(v[keep_rows], before[name][keep_rows])


def test_prompt_and_decode_steps():
    """Two requests: prompts of 300 and 517 tokens in one ragged append, then nine decode steps that append raw rows to
    the window rings, an entry whenever a block of four tokens completes, and attend."""
    import long_context_attention_compress_b200 as hca
    s = wl.PRO
    cfg = hca.make_cfg(s)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(8)
    lens, steps, B = [300, 517], 9, 2
    raw = [torch.randn(n + steps, s.c, generator=g).bfloat16() for n in lens]
    logits = [torch.randn(n + steps, s.c, generator=g).bfloat16() for n in lens]
    bias = (torch.randn(2 * s.m, s.c, generator=g) * 0.1).cuda()
    gamma = (torch.rand(s.c, generator=g) + 0.5).cuda()
    room = (max(lens) + steps) // s.m
    k = Cache("fp4", s.c, 64, B, room, rpb=32, seed=3)
    ring = Cache("bf16", s.c, 64, B, s.n_win, ring=True)
    ent = [hca.csa_compress(raw[b][:n].cuda(), logits[b][:n].cuda(), bias, s.m) for b, n in enumerate(lens)]
    cut = np.cumsum([0] + [e.shape[0] for e in ent])
    hca.kv_cache_append(torch.cat(ent), k.handle, i32([0, 0]), row_start=i32(cut), rate=s.m, gamma=gamma, rotate=True)
    rows0 = np.cumsum([0] + lens)
    hca.kv_cache_append(torch.cat([raw[b][:n] for b, n in enumerate(lens)]).cuda(), ring.handle, i32([0, 0]),
                        row_start=i32(rows0))
    for step in range(steps):
        pos = [n + step for n in lens]
        hca.kv_cache_append(torch.stack([raw[b][p] for b, p in enumerate(pos)]).cuda(), ring.handle, i32(pos))
        done = [(p + 1) // s.m - 1 if (p + 1) % s.m == 0 else -1 for p in pos]
        new = [hca.csa_compress(raw[b][max(0, p + 1 - 2 * s.m):p + 1].cuda(), logits[b][max(0, p + 1 - 2 * s.m):p + 1].cuda(),
                                bias, s.m)[-1:] for b, p in enumerate(pos)]
        hca.kv_cache_append(torch.cat(new), k.handle, i32(done), rate=s.m, gamma=gamma, rotate=True)
        q = torch.randn(B, s.n_heads, s.c, generator=g).bfloat16()
        win = ring.t["codes"]
        out = hca.sparse_mqa_attend_fp4(q.cuda(), k.handle, room, i32(pos), cfg, rate=s.m, win=win, rotate_out=True)
        back = to64(hca.kv_cache_gather(k.handle, B, room))
        for b, p in enumerate(pos):
            n = (p + 1) // s.m
            # every entry so far is the exact one's stored form, up to what the compressor's bf16 rounding may turn
            E = oracle.csa_compress(to64(raw[b][:p + 1]), to64(logits[b][:p + 1]), bias.double().cpu().numpy(), s.m)
            y = oracle.rope(oracle.rms_norm(oracle.round_bf16(E), gamma.double().cpu().numpy(), 1e-6),
                            oracle.entry_position(np.arange(n), s.m), 64, 10000.0)
            assert np.mean(np.abs(back[b, :n] - y) > 0.26 * np.abs(y) + 0.13 * np.abs(y).max(1, keepdims=True)) <= 1e-3
            rows = [raw[b][u] for u in range(max(0, p - s.n_win + 1), p + 1)]
            check_query(to64(out[b]), to64(q[b]), np.concatenate([back[b, :n], to64(torch.stack(rows))]), s.scale, None, p,
                        what=f"step {step} request {b}")
