"""Caches for the tests of the KV-cache operators: arrays of one form and
arrangement, the row an entry lives in, the rows an arrangement stands for
(float64, from the oracle's quantisers and value tables)."""

import numpy as np
import torch

import oracle
from parity_util import to64

BF16_HALF = 2.0 ** -8  # a rounding to bf16 is off by at most this, relative to the value


class Cache:
    """Arrays of `form` on the GPU, filled with recognisable bytes, behind a flat / paged / ring arrangement."""

    def __init__(self, form, c, rope_dims, n_req, room, rpb=0, ring=False, seed=0, fill=0x3C, spread=0):
        import long_context_attention_compress_b200 as hca
        self.form, self.c, self.rope, self.n_req, self.room, self.rpb, self.ring = form, c, rope_dims, n_req, room, rpb, ring
        self.table = None
        rng = np.random.default_rng(seed)
        if rpb:
            per = -(-room // rpb)
            blocks = n_req * per + 2
            self.table = torch.tensor(rng.permutation(blocks)[: n_req * per].reshape(n_req, per), dtype=torch.int32)
            lead = (blocks, rpb)
        else:
            lead = (n_req, room)
        n = c - rope_dims

        def arr(width, dtype, step):
            # rows `spread` steps of 16 bytes wider than needed
            w = width + spread * step
            b = torch.full((*lead, w * torch.empty((), dtype=dtype).element_size()), fill, dtype=torch.uint8)
            return b.view(dtype).cuda()
        if form == "bf16":
            self.t = {"codes": arr(c, torch.bfloat16, 8)}
        elif form == "fp8":
            self.t = {"codes": arr(n, torch.uint8, 16), "scales": arr(n // 64, torch.float32, 4)}
        else:
            self.t = {"codes": arr(n // 2, torch.uint8, 16), "scales": arr(-(-(n // 32) // 16) * 16, torch.uint8, 16)}
        if form != "bf16" and rope_dims:
            self.t["rope"] = arr(rope_dims, torch.bfloat16, 8)
        self.used = {"codes": c if form == "bf16" else n if form == "fp8" else n // 2,
                     "scales": n // (64 if form == "fp8" else 32), "rope": rope_dims}
        self.handle = hca.KvCache(form, c, rope_dims, **self.t,
                                  block_table=None if self.table is None else self.table.cuda(), ring=ring)

    def row(self, r, e):
        """Flat row number of entry e of request r."""
        if self.rpb:
            return int(self.table[r, e // self.rpb]) * self.rpb + e % self.rpb
        return r * self.room + (e % self.room if self.ring else e)

    def bytes(self):
        """{name: uint8 [rows, bytes of a row]} on the host (the part in use, then the rest)."""
        return {k: v.contiguous().view(torch.uint8).reshape(v.shape[0] * v.shape[1], -1).cpu().numpy()
                for k, v in self.t.items()}

    def width(self, name):
        return self.used[name] * self.t[name].element_size()


def stored(form, y, rope_dims):
    """Bytes of the stored form of rows y (float64, already what the form stores), by the oracle's quantisers."""
    n = y.shape[-1] - rope_dims
    bf = lambda v: torch.tensor(v).to(torch.bfloat16).view(torch.uint8).numpy().reshape(v.shape[0], -1)  # noqa: E731
    if form == "bf16":
        return {"codes": bf(y)}
    d = {"rope": bf(y[:, n:])} if rope_dims else {}
    if form == "fp4":
        codes, scales = oracle.mxfp4_quantize(y[:, :n])
        return {"codes": oracle.mxfp4_pack(codes), "scales": scales, **d}
    codes, scales, _ = oracle.fp8_kv_quantize(y, rope_dims)
    b = torch.tensor(codes).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # exact: E4M3 values
    return {"codes": b, "scales": scales.astype(np.float32).view(np.uint8).reshape(y.shape[0], -1), **d}


def values(form, bytes_, used, rope_dims):
    """float64 rows that bytes of a form stand for."""
    take = {k: np.ascontiguousarray(v[:, : used[k]]) for k, v in bytes_.items()}
    if form == "bf16":
        return to64(torch.tensor(take["codes"]).view(torch.bfloat16))
    if form == "fp4":
        v = oracle.mxfp4_dequantize(oracle.mxfp4_unpack(take["codes"]), take["scales"])
    else:
        v = oracle.fp8_kv_dequantize(to64(torch.tensor(take["codes"]).view(torch.float8_e4m3fn)),
                                     take["scales"].view(np.float32).astype(np.float64), np.zeros((v_len(take), 0)))
    if rope_dims:
        v = np.concatenate([v, to64(torch.tensor(take["rope"]).view(torch.bfloat16))], -1)
    return v


def v_len(take):
    return take["codes"].shape[0]


def fill_rows(cache, rows, y):
    """Store rows y (float64) at flat row numbers, from the host."""
    for k, b in stored(cache.form, y, cache.rope).items():
        flat = cache.t[k].view(torch.uint8).reshape(cache.t[k].shape[0] * cache.t[k].shape[1], -1)
        flat[torch.tensor(rows, device="cuda"), : b.shape[1]] = torch.tensor(b, device="cuda")
