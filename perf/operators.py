"""Cases of the KV-cache operators: appending rows to a cache, reading rows back, attending over a 4-bit cache.

The plain forms below are elementary torch operations on the operators' definitions (include/hca.h):
a row of c channels is stored as bf16, as FP8 (E4M3 codes, an f32 scale per 64 channels) or as FP4 (E2M1 codes,
a power-of-two scale per 32 channels), the last `rope` channels staying bf16; caches are flat, paged through a block
table, or rings.  Rows that are normalised and rotated on the way are computed in float64: they are then quantised,
and a value next to a rounding border must not fall on its other side.
"""

import math

import torch

own = False

DEV = "cuda"
EPS, BASE = 1e-6, 10000.0
N_WIN = 128


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one compressed entry for each of 8 requests at 1M tokens, straight from the compressor (f32), read back
        dict(name="append_entry_b8_fp4", op="append", form="fp4", c=512, rope=64, B=8, rows=8, most=8192, rpb=1, rate=128,
             f32=True, norm=True, ring=0, pad=0),
        # the raw rows of one decode step of 256 requests into their window rings
        dict(name="append_token_b256_ring", op="append", form="bf16", c=512, rope=64, B=256, rows=256, most=40000, rpb=0,
             rate=1, f32=False, norm=False, ring=128, pad=0),
        # ragged chunks of 13 requests into flat FP8 caches, behind them padding that is not appended
        dict(name="append_ragged_b13_fp8", op="append", form="fp8", c=512, rope=64, B=13, rows=3001, most=4096, rpb=0,
             rate=4, f32=True, norm=True, ring=0, pad=37),
        # the 16,384 entries of a 64K-token prompt into pages of 32, read back
        dict(name="append_prompt_64k_fp4", op="append", form="fp4", c=512, rope=64, B=1, rows=16384, most=16384, rpb=32,
             rate=4, f32=True, norm=True, ring=0, pad=0),
        # a chunk's entries in bf16 pages, queries' normalisation and rotation on the way
        dict(name="append_chunk_b4_bf16", op="append", form="bf16", c=512, rope=64, B=4, rows=4100, most=65536, rpb=32,
             rate=4, f32=False, norm=True, ring=0, pad=0),
        # indexer keys in 4 bits: 128 channels, no rotation, no normalisation, read back
        dict(name="append_keys_b3_fp4", op="append", form="fp4", c=128, rope=0, B=3, rows=24577, most=16384, rpb=32,
             rate=4, f32=False, norm=False, ring=0, pad=0),
        # every visible HCA entry of 8 requests at 1M tokens, widened
        dict(name="gather_all_b8_fp4", op="gather", form="fp4", c=512, rope=64, B=8, rows=8191, most=8192, rpb=1, sel=False),
        # the selected entries of one decode step, some slots empty
        dict(name="gather_sel_b32_fp8", op="gather", form="fp8", c=512, rope=64, B=32, rows=1024, most=4096, rpb=32, sel=True),
        # a short context, one request
        dict(name="attend_short_b1", op="attend", H=64, B=1, nq=1, N=129, k=0, rate=4, rpb=0, pos=517, sink=False, rot=False),
        # HCA decode of 8 requests at 1M tokens: 8,192 entries and the window
        dict(name="attend_hca_1m_b8", op="attend", H=64, B=8, nq=1, N=8192, k=0, rate=128, rpb=1, pos=1048575, sink=False,
             rot=False),
        # CSA decode of 32 requests at 128K tokens: 1,024 selected entries and the window, sinks, output rotated back
        dict(name="attend_csa_sel_b32", op="attend", H=64, B=32, nq=1, N=32768, k=1024, rate=4, rpb=32, pos=131071,
             sink=True, rot=True),
        # a chunk of queries of two requests over their cached entries, 16 heads (one of four shards)
        dict(name="attend_chunk_b2_h16", op="attend", H=16, B=2, nq=192, N=2900, k=0, rate=4, rpb=32, pos=11200, sink=True,
             rot=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attend", "attend", "attend"])
    if op == "append":
        form = rng.choice(["bf16", "fp8", "fp4"])
        c, rope = rng.choice([(512, 64), (512, 64), (512, 0), (128, 0), (256, 64)])
        B = _log(rng, 1, 64)
        rows = B if rng.random() < 0.4 else max(B, _log(rng, 64, 16384))
        ring = rng.choice([0, 0, 0, 128])
        rpb = 0 if ring else rng.choice([0, 1, 8, 32, 48])
        most = min(65536, max(rows, _log(rng, 256, 65536))) if not ring else _log(rng, 200, 100000)
        return dict(op=op, form=form, c=c, rope=rope, B=B, rows=rows, most=most if ring or B < 8 else min(most, 2048),
                    rpb=rpb, rate=rng.choice([1, 4, 128]), f32=rng.random() < 0.5, norm=rng.random() < 0.6, ring=ring,
                    pad=rng.choice([0, 0, 5]) if rows > B else 0)
    if op == "gather":
        B = _log(rng, 1, 32)
        most = _log(rng, 64, 8192)
        return dict(op=op, form=rng.choice(["bf16", "fp8", "fp4"]), c=512, rope=rng.choice([0, 64]), B=B,
                    rows=_log(rng, 1, most), most=most, rpb=rng.choice([0, 1, 16, 32]), sel=rng.random() < 0.5)
    H = rng.choice([64, 64, 64, 16, 32, 8, 128])
    rate = rng.choice([4, 4, 128])
    if rng.random() < 0.3:
        B, nq = rng.randint(1, 3), _log(rng, 2, 96)
        N = _log(rng, 16, 2048)
        k = 0
    else:
        B, nq = _log(rng, 1, 48), 1
        N = _log(rng, 1, max(2, min(32768, 131072 // B)))
        k = rng.choice([0, _log(rng, 1, 1024)])
        if not k:
            N = min(N, 8192)
    return dict(op=op, H=H, B=B, nq=nq, N=N, k=k, rate=rate, rpb=rng.choice([0, 1, 32, 40]),
                pos=max(nq - 1, N * rate - 1 + rng.randint(-2 * rate, 2 * rate)), sink=rng.random() < 0.5, rot=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ stored forms
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _fp4_codes(v):
    """MXFP4 of v [..., n] float64: (bytes [..., n/2], scale bytes [..., n/32])."""
    g = v.reshape(*v.shape[:-1], -1, 32)
    amax = g.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    a = torch.ldexp(g.abs(), -X)
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (m + 8 * ((g < 0) & (m > 0)).to(torch.uint8)).reshape(*v.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], (X[..., 0] + 127).to(torch.uint8)


def _fp8_codes(v):
    """E4M3 of v [..., n] float64: (bytes [..., n], f32 scales [..., n/64])."""
    g = v.reshape(*v.shape[:-1], -1, 64)
    amax = g.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax)).float()
    q = g / s.double()
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp_min(-5) - 4)
    r = (torch.round(q / step) * step).clamp(-448.0, 448.0)
    r = torch.copysign(r, q)
    return r.float().to(torch.float8_e4m3fn).view(torch.uint8).reshape(v.shape), s[..., 0]


def _store(form, y, rope):
    """The arrays of rows y (float64 of what is stored): a dict."""
    n = y.shape[-1] - rope
    if form == "bf16":
        return {"codes": y.float().to(torch.bfloat16)}
    codes, scales = (_fp4_codes if form == "fp4" else _fp8_codes)(y[..., :n])
    d = {"codes": codes, "scales": scales}
    if rope:
        d["rope"] = y[..., n:].float().to(torch.bfloat16)
    return d


def _values(form, d, dtype):
    """The rows that the arrays stand for."""
    if form == "bf16":
        return d["codes"].to(dtype)
    if form == "fp4":
        n = d["codes"].shape[-1] * 2
        t = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=DEV)
        v = t[torch.stack([d["codes"] & 15, d["codes"] >> 4], -1).reshape(*d["codes"].shape[:-1], n).int()]
        s = torch.ldexp(torch.ones((), dtype=dtype, device=DEV), d["scales"][..., : n // 32].int() - 127)
        v = (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)
    else:
        v = d["codes"].view(torch.float8_e4m3fn).to(dtype)
        v = (v.reshape(*v.shape[:-1], -1, 64) * d["scales"].to(dtype)[..., None]).reshape(v.shape)
    return torch.cat([v, d["rope"].to(dtype)], -1) if "rope" in d else v


def _empty(form, lead, c, rope):
    """Arrays for rows of the leading shape, as a program allocates them."""
    n = c - rope
    if form == "bf16":
        return {"codes": torch.zeros(*lead, c, dtype=torch.bfloat16, device=DEV)}
    d = {"codes": torch.zeros(*lead, n if form == "fp8" else n // 2, dtype=torch.uint8, device=DEV)}
    d["scales"] = (torch.ones(*lead, n // 64, device=DEV) if form == "fp8" else
                   torch.zeros(*lead, -(-(n // 32) // 16) * 16, dtype=torch.uint8, device=DEV))
    if rope:
        d["rope"] = torch.zeros(*lead, rope, dtype=torch.bfloat16, device=DEV)
    return d


def _put(arrays, rows, new):
    """arrays[rows] = new, on arrays [A, R, w] with flat row numbers."""
    for k, v in new.items():
        arrays[k].view(-1, arrays[k].shape[-1])[rows, : v.shape[-1]] = v


def _take(arrays, rows):
    return {k: v.view(-1, v.shape[-1])[rows] for k, v in arrays.items()}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(g, B, most, rpb):
    """A block table of shuffled blocks, and their number (a few of the pool's blocks belong to nobody)."""
    per = -(-most // rpb)
    n = B * per + 3
    return torch.randperm(n, generator=g, device=DEV)[: B * per].view(B, per).int(), n


def _rows_of(st, req, entry):
    """Flat row numbers of (request, entry) pairs."""
    req, entry = req.long(), entry.long()
    if st["ring"]:
        return req * st["ring"] + entry % st["ring"]
    if st["rpb"]:
        return st["table"][req, entry // st["rpb"]].long() * st["rpb"] + entry % st["rpb"]
    return req * st["most"] + entry


def _angles(pos, rope, dtype):
    j = torch.arange(rope // 2, device=DEV, dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(torch.tensor(BASE, dtype=torch.float64, device=DEV), -2.0 * j / rope)
    return torch.cos(a).to(dtype), torch.sin(a).to(dtype)


def _rotate(y, cs, sn, rope):
    """Pairs of the last `rope` channels of y turned by their angles."""
    n = y.shape[-1] - rope
    a, b = y[..., n::2], y[..., n + 1 :: 2]
    return torch.cat([y[..., :n], torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)], -1)


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "append":
        B, rows, c = case["B"], case["rows"], case["c"]
        x = torch.randn(rows + case["pad"], c, generator=g, device=DEV)
        st["x"] = x if case["f32"] else x.to(torch.bfloat16)
        if rows > B:  # ragged: at least one row a request
            cut = torch.rand(B - 1, generator=g, device=DEV).mul(rows - B + 1).long().sort()[0] + torch.arange(1, B, device=DEV)
            st["start"] = torch.cat([torch.zeros(1, device=DEV), cut, torch.full((1,), rows, device=DEV)]).int()
            count = st["start"][1:] - st["start"][:-1]
        else:
            st["start"], count = None, torch.ones(B, dtype=torch.int32, device=DEV)
        # the first new entry of each request: the new rows end at or before `most` (a prompt's begin at 0)
        if not case["ring"]:
            st["most"] = max(case["most"], int(count.max()))
        room = (st["most"] - count).clamp_min(0) * (B > 1 or rows == 1)
        st["first"] = torch.minimum((torch.rand(B, generator=g, device=DEV) * (room + 1)).int(), room.int())
        st["gamma"] = torch.rand(c, generator=g, device=DEV) + 0.5 if case["norm"] else None
    elif case["op"] == "gather":
        st["ring"] = 0
        if case["sel"]:
            st["idx"] = torch.randint(-1, case["most"], (case["B"], case["rows"]), generator=g, device=DEV).int()
    else:
        B, nq, H, c, k = case["B"], case["nq"], case["H"], 512, case["k"]
        st |= dict(ring=0, most=case["N"], form="fp4", c=c, rope=64)
        st["q"] = torch.randn(B * nq, H, c, generator=g, device=DEV).to(torch.bfloat16)
        # the queries of a request end at `pos` less a little, one after the other
        last = case["pos"] - torch.randint(0, max(1, min(case["rate"], case["pos"] - nq + 2)), (B,), generator=g, device=DEV)
        st["q_pos"] = (last[:, None] - (nq - 1) + torch.arange(nq, device=DEV)).clamp_min(0).flatten().int()
        st["q_req"] = torch.arange(B, device=DEV).repeat_interleave(nq).int() if nq > 1 else None
        st["W"] = N_WIN if nq == 1 else N_WIN + nq - 1
        st["win"] = torch.randn(B, st["W"], c, generator=g, device=DEV).to(torch.bfloat16)
        st["sink_l"] = torch.randn(H, generator=g, device=DEV) if case["sink"] else None
        if k:  # k of the visible entries in no order, -1 where there are fewer
            vis = ((st["q_pos"].long() + 1) // case["rate"]).clamp_max(case["N"])
            key = torch.rand(B, case["N"], generator=g, device=DEV)
            key[torch.arange(case["N"], device=DEV)[None] >= vis[:, None]] = -1.0
            top, at = key.topk(min(k, case["N"]), -1)
            at = torch.where(top >= 0, at, -1).int()
            st["idx"] = torch.nn.functional.pad(at, (0, k - at.shape[1]), value=-1).contiguous()
    if st["ring"]:
        lead = (st["B"], st["ring"])
    elif st["rpb"]:
        st["table"], blocks = _table(g, st["B"], st["most"], st["rpb"])
        lead = (blocks, st["rpb"])
    else:
        lead = (st["B"], st["most"])
    st["arrays"] = _empty(st["form"], lead, st["c"], st["rope"])
    if case["op"] != "append":  # what the cache holds: rows of unit variance
        rows = torch.arange(lead[0] * lead[1], device=DEV)
        for part in rows.split(65536):
            y = torch.randn(part.numel(), st["c"], generator=g, device=DEV).to(torch.bfloat16).double()
            _put(st["arrays"], part, _store(st["form"], y, st["rope"]))
    if own:  # the handle and the workspace that a program keeps beside its cache
        import long_context_attention_compress_b200 as hca
        from types import SimpleNamespace

        st["cache"] = hca.KvCache(st["form"], st["c"], st["rope"], **st["arrays"], block_table=st.get("table"),
                                  ring=bool(st["ring"]))
        if case["op"] == "attend":
            st["cfg"] = hca.make_cfg(SimpleNamespace(c=512, m=4, m_hca=128, topk=max(1, case["k"]), n_idx_heads=64, d_idx=128,
                                                     n_heads=case["H"], n_win=N_WIN, scale=512 ** -0.5, rope_dims=64,
                                                     rope_base=BASE, norm_eps=EPS))
            st["ws"] = torch.empty(max(1, hca.sparse_mqa_attend_fp4_workspace(st["cfg"], case["B"] * case["nq"], case["N"],
                                                                              case["k"])), dtype=torch.uint8, device=DEV)
    return st


def _new_rows(st):
    """(request, entry) of each appended row, and whether a ring keeps it."""
    n = st["rows"]
    i = torch.arange(n, device=DEV)
    if st["start"] is None:
        req, j, count = i, torch.zeros_like(i), torch.ones_like(i)
    else:
        req = torch.searchsorted(st["start"].long(), i, right=True) - 1
        j = i - st["start"].long()[req]
        count = (st["start"][1:] - st["start"][:-1]).long()[req]
    return req, st["first"].long()[req] + j, (j >= count - st["ring"]) if st["ring"] else torch.ones_like(i, dtype=torch.bool)


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    return {"append": _append, "gather": _gather, "attend": _attend}[st["op"]](st)


def _append(st):
    a, rope = st["arrays"], st["rope"]
    if own:
        import long_context_attention_compress_b200 as hca

        hca.kv_cache_append(st["x"], st["cache"], st["first"], row_start=st["start"], rate=st["rate"], gamma=st["gamma"],
                            rotate=st["norm"], norm_eps=EPS, rope_base=BASE)
    else:
        req, entry, kept = _new_rows(st)
        y = st["x"][: st["rows"]].double()
        if st["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["gamma"].double()
            if rope:
                y = _rotate(y, *_angles((entry + 1) * st["rate"] - 1, rope, torch.float64), rope)
            y = y.float().to(torch.bfloat16).double()
        rows = _rows_of(st, req, entry)
        _put(a, rows[kept], {k: v[kept] for k, v in _store(st["form"], y, rope).items()})
    if st["form"] == "bf16":
        return {"rows": a["codes"]}
    if st["form"] == "fp8":
        return {"codes": a["codes"].view(torch.float8_e4m3fn), "scales": a["scales"], "rope": a.get("rope")}
    # 4 bits: the new rows (a ring: all of it) read back as the values that they stand for
    if own:
        if st["ring"]:
            return {"rows": hca.kv_cache_gather(st["cache"], st["B"], st["ring"])}
        most = st["rows"] if st["B"] == 1 else 1 if st["start"] is None else -(-st["rows"] // st["B"])
        return {"rows": hca.kv_cache_gather(st["cache"], st["B"], most, first=st["first"])}
    r = torch.arange(st["B"], device=DEV)
    if st["ring"]:
        return {"rows": _values("fp4", {k: v[..., : (st["c"] - rope) // 32] if k == "scales" else v for k, v in a.items()},
                                torch.float32).to(torch.bfloat16)}
    most = st["rows"] if st["B"] == 1 else 1 if st["start"] is None else -(-st["rows"] // st["B"])
    e = st["first"].long()[:, None] + torch.arange(most, device=DEV)
    ok = e < st["most"]
    v = _values("fp4", _take(a, _rows_of(st, r[:, None].expand_as(e), e.clamp_max(st["most"] - 1))), torch.float32)
    return {"rows": torch.where(ok[..., None], v, 0.0).to(torch.bfloat16)}


def _gather(st):
    if own:
        import long_context_attention_compress_b200 as hca

        return hca.kv_cache_gather(st["cache"], st["B"], st["rows"], idx=st.get("idx"))
    e = st["idx"].long() if st["sel"] else torch.arange(st["rows"], device=DEV)[None].expand(st["B"], -1)
    r = torch.arange(st["B"], device=DEV)[:, None].expand_as(e)
    v = _values(st["form"], _take(st["arrays"], _rows_of(st, r, e.clamp_min(0))), torch.float32)
    return torch.where((e >= 0)[..., None], v, 0.0).to(torch.bfloat16)


def _attend(st):
    if own:
        import long_context_attention_compress_b200 as hca

        return hca.sparse_mqa_attend_fp4(st["q"], st["cache"], st["N"], st["q_pos"], st["cfg"], idx=st.get("idx"),
                                         rate=st["rate"], win=st["win"], q_req=st["q_req"], sink=st["sink_l"],
                                         rotate_out=st["rot"], ws=st["ws"])
    B, nq, H, N, W, c = st["B"], st["nq"], st["H"], st["N"], st["W"], st["c"]
    pos = st["q_pos"].long()
    r = torch.arange(B, device=DEV)
    q = st["q"].float().view(B, nq * H, c) * c ** -0.5
    if st["k"]:
        e = st["idx"].long()
        ok = (e >= 0).view(B, 1, 1, -1)
        e = e.clamp_min(0)
    else:
        e = torch.arange(N, device=DEV)[None].expand(B, N)
        ok = (e[0][None] < ((pos + 1) // st["rate"]).clamp_max(N)[:, None]).view(B, nq, 1, N)
    rows = _values("fp4", _take(st["arrays"], _rows_of(st, r[:, None].expand_as(e), e)), torch.float32)  # [B, R, c]
    # window: token tau of a request is row tau % W of its ring
    slot = torch.arange(W, device=DEV)
    age = (pos[:, None] - slot) % W  # tokens back from the query
    wok = ((age < N_WIN) & (age <= pos[:, None])).view(B, nq, 1, W)
    rows = torch.cat([rows, st["win"].float()], 1)
    ok = torch.cat([ok.expand(B, nq, 1, rows.shape[1] - W), wok], -1)
    s = torch.bmm(q, rows.transpose(1, 2)).view(B, nq, H, -1).masked_fill(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    if st["sink_l"] is not None:
        m = torch.maximum(m, st["sink_l"].view(1, 1, H, 1))
    p = torch.exp(s - m)
    den = p.sum(-1, keepdim=True)
    if st["sink_l"] is not None:
        den = den + torch.exp(st["sink_l"].view(1, 1, H, 1) - m)
    o = (torch.bmm(p.view(B, nq * H, -1), rows).view(B, nq, H, c) / den).view(B * nq, H, c)
    if st["rot"]:
        cs, sn = _angles(pos, 64, torch.float32)
        o = _rotate(o, cs[:, None], -sn[:, None], 64)
    return o.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def _row_bytes(form, c, rope):
    n = c - rope
    return 2 * c if form == "bf16" else n + n // 64 * 4 + 2 * rope if form == "fp8" else n // 2 + n // 32 + 2 * rope


def work(case):
    if case["op"] == "append":
        n = case["rows"]
        back = n * case["c"] * 2 if case["form"] == "fp4" else 0
        return {"bytes": n * (case["c"] * (4 if case["f32"] else 2) + _row_bytes(case["form"], case["c"], case["rope"])) + back,
                "flops": 0}
    if case["op"] == "gather":
        n = case["B"] * case["rows"]
        return {"bytes": n * (_row_bytes(case["form"], case["c"], case["rope"]) + 2 * case["c"]), "flops": 0}
    B, nq, H = case["B"], case["nq"], case["H"]
    seen = min(case["k"] or case["N"], (case["pos"] + 1) // case["rate"])
    win = min(N_WIN, case["pos"] + 1)
    return {"bytes": B * (seen * _row_bytes("fp4", 512, 64) + (win + nq - 1) * 1024) + 2 * B * nq * H * 1024,
            "flops": 4.0 * B * nq * H * 512 * (seen + win)}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits
def _e2m1_nearest(a):
    """Nearest E2M1 magnitude of a >= 0 (float64), the even code on a tie: by distances."""
    t = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    d = (a.clamp_max(6.0)[..., None] - t).abs()
    odd = torch.tensor([0, 1] * 4, dtype=torch.float64, device=DEV) * 1e-13
    return t[(d + odd).argmin(-1)]


def _exact_row(form, y, rope):
    """What a row y (float64) reads as once stored, and the FP8 codes and scales apart."""
    n = y.shape[-1] - rope
    tail = y[:, n:].float().to(torch.bfloat16).double()
    head = y[:, :n]
    if form == "bf16":
        return y.float().to(torch.bfloat16).double(), None, None
    if form == "fp4":
        g = head.reshape(y.shape[0], -1, 32)
        top = g.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top.clamp_min(1e-300))) - 2), torch.ones_like(top))
        parts = [torch.copysign(_e2m1_nearest((p / q).abs()) * q, p) for p, q in zip(g.split(2048), s.split(2048))]
        return torch.cat([torch.cat(parts).reshape(head.shape), tail], -1), None, None
    g = head.reshape(y.shape[0], -1, 64)
    top = g.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, top / 448, torch.ones_like(top)).float().double()
    q = g / s
    ulp = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    low = torch.floor(q / ulp)
    rest = q / ulp - low
    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))
    code = ((low + up) * ulp).clamp(-448, 448)
    return torch.cat([(code * s).reshape(head.shape), tail], -1), code.reshape(head.shape), s[..., 0]


def exact(case, seed):
    st = prepare(case, seed)
    c, rope = st["c"], st["rope"]
    if case["op"] == "append":
        i = torch.arange(case["rows"], device=DEV)
        start = st["start"].long() if st["start"] is not None else torch.arange(case["B"] + 1, device=DEV)
        req = (i[:, None] >= start[None, 1:]).sum(1)
        entry = st["first"].long()[req] + i - start[req]
        last = st["first"].long()[req] + start[req + 1] - start[req] - 1
        y = st["x"][: case["rows"]].double()
        if case["norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c + EPS) * st["gamma"].double()
            if rope:
                j = torch.arange(rope // 2, dtype=torch.float64, device=DEV)
                ang = ((entry + 1) * case["rate"] - 1).double()[:, None] * BASE ** (-2 * j / rope)
                z = torch.view_as_complex(y[:, c - rope :].reshape(-1, rope // 2, 2).contiguous())
                z = z * torch.polar(torch.ones_like(ang), ang)
                y = torch.cat([y[:, : c - rope], torch.view_as_real(z).flatten(1)], -1)
            y = y.float().to(torch.bfloat16).double()
        keep = entry > last - st["ring"] if st["ring"] else entry >= 0
        v, codes, scales = _exact_row(st["form"], y[keep], rope)
        req, entry = req[keep], entry[keep]
        if st["form"] == "fp4" and not st["ring"]:
            most = case["rows"] if case["B"] == 1 else 1 if st["start"] is None else -(-case["rows"] // case["B"])
            out = torch.zeros(case["B"], most, c, dtype=torch.float64, device=DEV)
            at = entry - st["first"].long()[req]
            out[req[at < most], at[at < most]] = v[at < most]
            return {"rows": out}
        where = (req, entry % st["ring"]) if st["ring"] else (
            (st["table"].long()[req, entry // st["rpb"]], entry % st["rpb"]) if st["rpb"] else (req, entry))
        lead = st["arrays"]["codes"].shape[:2]

        def full(w, new, fill=0.0):
            o = torch.full((*lead, w), fill, dtype=torch.float64, device=DEV)
            o[where] = new
            return o

        if st["form"] == "fp8":
            return {"codes": full(c - rope, codes), "scales": full((c - rope) // 64, scales, 1.0),
                    "rope": full(rope, v[:, c - rope :]) if rope else None}
        return {"rows": full(c, v)}
    if case["op"] == "gather":
        return _gather_exact(st)
    return _attend_exact(st)


def _stored(st, req, entry):
    """Row values (float64) of one request's entries."""
    if st["rpb"]:
        b, o = st["table"].long()[req][entry // st["rpb"]], entry % st["rpb"]
    else:
        b, o = torch.full_like(entry, req), entry
    a = {k: v[b, o] for k, v in st["arrays"].items()}
    n = st["c"] - st["rope"]
    if st["form"] == "bf16":
        return a["codes"].double()
    if st["form"] == "fp8":
        v = a["codes"].view(torch.float8_e4m3fn).double() * a["scales"].double().repeat_interleave(64, -1)
    else:
        code = torch.empty(entry.numel(), n, dtype=torch.long, device=DEV)
        code[:, 0::2], code[:, 1::2] = (a["codes"] % 16).long(), (a["codes"] // 16).long()
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[code % 8]
        v = torch.where(code >= 8, -mag, mag) * torch.exp2(a["scales"][:, : n // 32].double() - 127).repeat_interleave(32, -1)
    return torch.cat([v, a["rope"].double()], -1) if st["rope"] else v


def _gather_exact(st):
    out = torch.zeros(st["B"], st["rows"], st["c"], dtype=torch.float64, device=DEV)
    for b in range(st["B"]):
        e = st["idx"][b].long() if st["sel"] else torch.arange(st["rows"], device=DEV)
        out[b][e >= 0] = _stored(st, b, e[e >= 0])
    return out


def _attend_exact(st):
    H, c = st["H"], st["c"]
    out = torch.zeros(st["B"] * st["nq"], H, c, dtype=torch.float64, device=DEV)
    for b in range(st["B"]):
        every = None if st["k"] else _stored(st, b, torch.arange(st["N"], device=DEV))
        for i in range(st["nq"]):
            t = b * st["nq"] + i
            p = int(st["q_pos"][t])
            if st["k"]:
                e = st["idx"][t].long()
                rows = _stored(st, b, e[e >= 0])
            else:
                rows = every[: min(st["N"], (p + 1) // st["rate"])]
            tok = torch.arange(max(0, p - N_WIN + 1), p + 1, device=DEV)
            rows = torch.cat([rows, st["win"][b][tok % st["W"]].double()])
            s = st["q"][t].double() @ rows.T / math.sqrt(c)
            if st["sink_l"] is not None:
                s = torch.cat([s, st["sink_l"].double()[:, None]], -1)
            o = torch.softmax(s, -1)[:, : rows.shape[0]] @ rows
            if st["rot"]:
                ang = -p * BASE ** (-2 * torch.arange(32, dtype=torch.float64, device=DEV) / 64)
                z = torch.view_as_complex(o[:, c - 64 :].reshape(H, 32, 2).contiguous()) * torch.polar(torch.ones_like(ang), ang)
                o = torch.cat([o[:, : c - 64], torch.view_as_real(z).flatten(1)], -1)
            out[t] = o
    return out
