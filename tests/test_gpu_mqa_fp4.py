"""sparse_mqa_attend_fp4 on the GPU against float64 attention over the rows that the cache's bytes stand for.

Tolerance.  With p the exact probabilities, an output element is
o = sum_u p_u row_u, and the kernel's differs by
  - each p_u's own error d_u, |d_u| <= 2^-8 (rounded to bf16; the denominator is the sum of the rounded ones) + 2 e_s,
    e_s = 520 * 2^-24 * scale * sum_d |q_d row_d|, the f32 logit's: at most max|d| * (sum p|row| + |o|);
  - f32 sums over U rows: U * 2^-23 * sum p|row|;
  - the output's rounding to bf16: 2^-8 |o|.
The bound is taken element by element (rotated like the output where it is rotated back).  Rows are random, so the
errors of the rows are independent and add up as the rows themselves do: the 2-norm of the error over a query's
output is also held to 2^-7 of the output's."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import BF16_HALF, Cache, fill_rows, values
from parity_util import to64
from types import SimpleNamespace

pytestmark = pytest.mark.gpu
BASE = 10000.0


def make(c, H, n_win=128, rope=64, m=4):
    import long_context_attention_compress_b200 as hca
    return hca.make_cfg(SimpleNamespace(c=c, m=m, m_hca=128, topk=1024, n_idx_heads=64, d_idx=128, n_heads=H, n_win=n_win,
                                        scale=c ** -0.5, rope_dims=rope, rope_base=BASE, norm_eps=1e-6))


def check_query(got, q, rows, scale, sink=None, rotate_by=None, rope=64, what=""):
    """One query's output [H, c] against the definition, within the bounds derived above."""
    c = q.shape[1]
    z = None if sink is None else np.asarray(sink, dtype=np.float64)
    o = oracle.mqa_attend(q, rows, scale, z)
    s = scale * (q @ rows.T)
    m = s.max(1, keepdims=True) if z is None else np.maximum(s.max(1, keepdims=True), z[:, None])
    p = np.exp(s - m)
    p /= p.sum(1, keepdims=True) + (0 if z is None else np.exp(z[:, None] - m))
    mass = p @ np.abs(rows)
    e_s = 520 * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(rows).T).max(1, keepdims=True)
    bound = (BF16_HALF + 2 * e_s) * (mass + np.abs(o)) + len(rows) * 2.0 ** -23 * mass
    if rotate_by is not None:
        o = oracle.rope(o, -rotate_by, rope, BASE)
        cs = np.abs(np.cos(rotate_by * oracle.rope_theta(rope, BASE)))
        sn = np.abs(np.sin(rotate_by * oracle.rope_theta(rope, BASE)))
        n = c - rope
        a, b = bound[:, n::2].copy(), bound[:, n + 1::2].copy()
        bound[:, n::2], bound[:, n + 1::2] = a * cs + b * sn, a * sn + b * cs
    bound += BF16_HALF * np.abs(o) + 1e-30
    err = np.abs(got - o)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))
    assert np.linalg.norm(err) <= 2.0 ** -7 * np.linalg.norm(o) + 1e-30, (what, np.linalg.norm(err) / np.linalg.norm(o))


class Setup:
    def __init__(self, c=512, rope=64, H=64, B=2, N=300, rpb=0, nq=1, n_win=128, W=None, seed=0, spread=0, scale=1.0,
                 win=True):
        rng = np.random.default_rng(seed)
        self.c, self.rope, self.H, self.B, self.N, self.nq, self.n_win = c, rope, H, B, N, nq, n_win
        self.k = Cache("fp4", c, rope, B, max(1, N), rpb=rpb, seed=seed, fill=0xFF, spread=spread)
        if N:
            rows = [self.k.row(b, e) for b in range(B) for e in range(N)]
            fill_rows(self.k, rows, to64(torch.tensor(rng.normal(size=(B * N, c)) * scale).bfloat16()))
        self.ref = values("fp4", self.k.bytes(), {n: self.k.width(n) for n in self.k.t}, rope)
        self.q = torch.tensor(rng.normal(size=(B * nq, H, c))).bfloat16()
        self.W = W or n_win + nq - 1
        self.win = torch.tensor(rng.normal(size=(B, self.W, c)) * scale).bfloat16() if win else None
        self.cfg = make(c, H, n_win, rope)

    def call(self, q_pos, rate=4, idx=None, q_req=None, sink=None, rotate=False, N=None, **kw):
        import long_context_attention_compress_b200 as hca
        i32 = lambda v: None if v is None else torch.tensor(np.asarray(v), dtype=torch.int32).cuda()  # noqa: E731
        return hca.sparse_mqa_attend_fp4(
            self.q.cuda(), self.k.handle, self.N if N is None else N, i32(q_pos), self.cfg, idx=i32(idx), rate=rate,
            win=None if self.win is None else self.win.cuda(), q_req=i32(q_req),
            sink=None if sink is None else torch.tensor(sink, dtype=torch.float32).cuda(), rotate_out=rotate, **kw)

    def rows(self, i, t, r, rate, idx, N=None):
        N = self.N if N is None else N
        if t < 0 or not 0 <= r < self.B:
            return np.zeros((0, self.c))
        e = [s for s in (idx[i] if idx is not None else range(min(N, (t + 1) // rate))) if 0 <= s < N]
        out = [self.ref[self.k.row(r, int(s))] for s in e]
        if self.win is not None:
            out += [to64(self.win[r, tok % self.W]) for tok in range(max(0, t - self.n_win + 1), t + 1)]
        return np.array(out).reshape(-1, self.c)

    def check(self, got, q_pos, rate=4, idx=None, q_req=None, sink=None, rotate=False, N=None):
        got = to64(got)
        assert got.shape == tuple(self.q.shape)
        for i, t in enumerate(np.asarray(q_pos)):
            t, r = int(t), int(i if q_req is None else q_req[i])
            rows = self.rows(i, t, r, rate, idx, N)
            if not len(rows):
                assert not got[i].any(), f"query {i} has no rows"
                continue
            check_query(got[i], to64(self.q[i]), rows, self.cfg.scale, sink, t if rotate else None, self.rope, f"query {i}")


@pytest.mark.parametrize("H", [64, 1, 4, 16, 40, 128])
@pytest.mark.parametrize("rpb", [0, 1, 32])
def test_dense_heads(H, rpb):
    s = Setup(H=H, rpb=rpb, N=333)
    pos = [1331, 900]
    s.check(s.call(pos), pos)


@pytest.mark.parametrize("N,pos", [(0, [0, 5]), (1, [3, 2]), (1, [4, 130]), (31, [123, 127]), (127, [508, 511]),
                                   (128, [511, 512]), (129, [515, 516]), (257, [1027, 700]), (1000, [3999, 3])])
def test_dense_lengths(N, pos):
    """Lengths around the 128-row tile, windows shorter than n_win, entries not visible yet."""
    s = Setup(N=N, rpb=8, seed=N)
    s.check(s.call(pos), pos)


@pytest.mark.parametrize("n_win,W", [(1, 1), (7, 9), (128, 128), (200, 256), (128, 5000)])
def test_windows(n_win, W):
    s = Setup(N=64, n_win=n_win, W=W, seed=n_win)
    pos = [259, 4200]
    s.check(s.call(pos), pos)


def test_no_window_and_no_rows():
    """Without a window a query before the first entry has no rows: zeros, with a sink too; padding queries likewise."""
    s = Setup(N=300, win=False)
    for sink in (None, np.linspace(-2, 2, 64)):
        pos = [2, 800]
        s.check(s.call(pos, sink=sink), pos, sink=sink)
        pos = [-1, -7]
        got = s.call(pos, sink=sink)
        assert not got.any()
    idx = np.full((2, 64), -1)
    pos = [800, 801]
    s.check(s.call(pos, idx=idx), pos, idx=idx)
    idx[1, 17] = 5
    s.check(s.call(pos, idx=idx), pos, idx=idx)


@pytest.mark.parametrize("k", [1, 100, 128, 1000, 1024])
@pytest.mark.parametrize("rpb", [0, 32])
def test_selected(k, rpb):
    """Selected entries with empty and out-of-range slots, and one selected twice (it counts twice)."""
    s = Setup(B=3, N=2048, rpb=rpb, seed=k)
    rng = np.random.default_rng(k)
    idx = np.stack([rng.permutation(2048)[:k] for _ in range(3)])
    if k > 4:
        idx[0, : k // 2] = -1
        idx[1, 3] = 2048
        idx[1, 4] = idx[1, 2]
        idx[2, -1] = -5
    pos = [8191, 8191, 8200]
    s.check(s.call(pos, idx=idx), pos, idx=idx)


@pytest.mark.parametrize("H,sink,rotate", [(64, True, True), (64, False, True), (16, True, False), (100, True, True)])
@pytest.mark.parametrize("N", [100, 3000])
def test_sink_and_rotation(H, sink, rotate, N):
    """Split and unsplit queries; sinks far above and below the logits."""
    s = Setup(H=H, N=N, rpb=32, seed=H)
    z = np.random.default_rng(1).normal(size=H) * 3 if sink else None
    if sink:
        z[0], z[1 % H] = 12.0, -50.0
    pos = [4 * N - 1, 4 * N + 77]
    s.check(s.call(pos, sink=z, rotate=rotate), pos, sink=z, rotate=rotate)


@pytest.mark.parametrize("nq,H", [(3, 64), (37, 16)])
def test_several_queries_a_request(nq, H):
    """Chunks of queries of two requests; one query without a request, one before the sequence."""
    s = Setup(H=H, B=2, N=200, rpb=16, nq=nq, seed=nq)
    req = np.repeat([1, 0], nq)
    pos = np.concatenate([700 + np.arange(nq), 130 + np.arange(nq)])
    s.check(s.call(pos, q_req=req, rotate=True), pos, q_req=req, rotate=True)
    req[0], pos[-1], req[1] = 2, -3, -1
    s.check(s.call(pos, q_req=req), pos, q_req=req)


@pytest.mark.parametrize("H,nq", [(1, 70), (2, 33), (5, 29), (7, 13), (16, 21), (24, 9), (32, 5)])
@pytest.mark.parametrize("N", [90, 700])
def test_queries_that_share_columns(H, nq, N):
    """Few heads: the columns of one CTA belong to several queries, whose requests and positions change inside it."""
    s = Setup(H=H, B=3, N=N, rpb=16, nq=nq, W=700, seed=H)
    rng = np.random.default_rng(H)
    req = np.repeat([2, 0, 1], nq)
    pos = np.concatenate([4 * N - 3 - nq + np.arange(nq), 40 + np.arange(nq), 200 + np.arange(nq)])
    z = rng.normal(size=H)
    s.check(s.call(pos, q_req=req, rotate=True, sink=z), pos, q_req=req, rotate=True, sink=z)
    # any order of requests, positions far apart and equal, padding queries in between
    req = rng.integers(0, 3, 3 * nq)
    req[nq // 2: nq // 2 + 6] = 1
    pos = rng.integers(0, 4 * N + 50, 3 * nq)
    pos[nq // 2: nq // 2 + 6] = [300, 303, 299, 299, 304, 309]
    pos[5], req[8] = -1, 3
    s.check(s.call(pos, q_req=req), pos, q_req=req)
    s.win = None
    s.check(s.call(pos, q_req=req, sink=z), pos, q_req=req, sink=z)


def test_one_query_a_request_named():
    """q_req names the same requests as its absence, in another order, for one query each."""
    s = Setup(H=8, B=5, N=300, rpb=0, seed=4)
    pos = np.array([1199, 700, 3, 1100, 1000])
    s.check(s.call(pos, q_req=np.arange(5)), pos, q_req=np.arange(5))
    req = np.array([3, 1, 4, 0, 2])
    s.check(s.call(pos, q_req=req), pos, q_req=req)


def test_many_queries_unsplit():
    """More queries than the machine has room for: one CTA walks all of a query's rows."""
    s = Setup(H=64, B=1, N=600, nq=400, seed=3)
    pos = 2000 + np.arange(400)
    req = np.zeros(400, int)
    got = s.call(pos, q_req=req)
    keep = [0, 1, 199, 399]
    sub = Setup.__new__(Setup)
    sub.__dict__ = dict(s.__dict__, q=s.q[keep])
    sub.check(got[keep], pos[keep], q_req=req[keep])


@pytest.mark.parametrize("H", [4, 16, 64])
@pytest.mark.parametrize("where", ["entry", "window"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_rows_that_earlier_queries_do_not_see(H, where, value):
    """Queries of one chunk: a row that is not finite reaches the queries that see it and no other."""
    s = Setup(H=H, B=1, N=300, nq=4, seed=H)
    pos = np.array([601, 602, 603, 604])  # rate 4: 150 entries are visible to the first two, 151 to the others
    first, clean = 2, s.win.clone()
    if where == "entry":
        s.k.t["rope"].view(-1, s.k.t["rope"].shape[-1])[s.k.row(0, 150), 5] = value
    else:
        s.win[0, 603 % s.W, 17] = value
    out = s.call(pos, q_req=[0] * 4)
    s.win = clean
    got = to64(out)
    assert np.isfinite(got[:first]).all()
    for i in range(first):
        check_query(got[i], to64(s.q[i]), s.rows(i, int(pos[i]), 0, 4, None), s.cfg.scale, what=f"query {i}")
    if np.isnan(value):
        assert np.isnan(got[first:]).all()
    else:
        assert (~np.isfinite(got[first:])).any(axis=(1, 2)).all()


@pytest.mark.parametrize("c,rope,H", [(64, 0, 4), (64, 32, 4), (128, 64, 8), (256, 0, 64), (480, 64, 3), (512, 0, 64),
                                      (512, 256, 64)])
def test_other_widths(c, rope, H):
    s = Setup(c=c, rope=rope, H=H, N=150, rpb=8, n_win=32, seed=c)
    pos = [599, 610]
    s.check(s.call(pos), pos)


@pytest.mark.parametrize("scale", [1e-20, 1e-3, 30.0])
def test_magnitudes(scale):
    """Tiny rows (all logits equal), and large ones (the softmax picks single rows, running maxima move)."""
    s = Setup(N=700, scale=scale, seed=5)
    pos = [2799, 2000]
    s.check(s.call(pos), pos)


def test_ascending_logits_rescale():
    """Logits that grow along the row list: the running maximum moves at every tile."""
    import long_context_attention_compress_b200 as hca  # noqa: F401
    s = Setup(N=1024, seed=6, win=False)
    u = to64(torch.tensor(np.random.default_rng(0).normal(size=512)).bfloat16())
    y = np.stack([to64(torch.tensor(u * (0.02 + 2.0 * e / 1024)).bfloat16()) for e in range(1024)])
    for b in range(2):
        fill_rows(s.k, [s.k.row(b, e) for e in range(1024)], y)
    s.ref = values("fp4", s.k.bytes(), {n: s.k.width(n) for n in s.k.t}, 64)
    s.q = torch.tensor(np.broadcast_to(u * 2, (2, 64, 512)).copy() * np.linspace(0.1, 1, 64)[None, :, None]).bfloat16()
    pos = [4095, 3000]
    s.check(s.call(pos), pos)


def test_spread_rows_and_garbage_outside():
    """Row strides wider than the row; bytes of unused rows and blocks are 0xFF (NaN scales, NaN rope): never used."""
    s = Setup(N=77, rpb=16, spread=3, B=3, seed=8)
    pos = [307, 200, 3]
    s.check(s.call(pos), pos)


def test_split_and_unsplit_agree_and_repeat():
    """The same bits again, and the same bits with a larger workspace than needed."""
    s = Setup(N=5000, B=2, seed=9)
    pos = [19999, 15000]
    a = s.call(pos)
    s.check(a, pos)
    for _ in range(3):
        assert torch.equal(a, s.call(pos))
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, s.call(pos, ws=ws))


def test_other_stream_and_graph():
    import long_context_attention_compress_b200 as hca
    s = Setup(N=900, B=2, rpb=32, seed=10)
    pos = [3599, 3000]
    want = s.call(pos)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = s.call(pos, stream=st)
    st.synchronize()
    assert torch.equal(want, got)
    q, win = s.q.cuda(), s.win.cuda()
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(hca.sparse_mqa_attend_fp4_workspace(s.cfg, 2, 900), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hca.sparse_mqa_attend_fp4(q, s.k.handle, 900, p, s.cfg, rate=4, win=win, out=out, ws=ws)
    g.replay()
    assert torch.equal(want, out)
    p[0] = 1000
    g.replay()
    s.check(out, [1000, 3000])


def test_index_check(monkeypatch):
    """HCA_DEBUG=1: entries out of range, not visible yet, and blocks outside the pool are recorded."""
    import long_context_attention_compress_b200 as hca
    s = Setup(N=256, B=1, rpb=32, seed=11)
    assert hca.lib.hca_check_device() == 0, hca.last_error()
    monkeypatch.setenv("HCA_DEBUG", "1")
    ok = np.arange(64)[None]
    s.call([1023], idx=ok)
    assert hca.lib.hca_check_device() == 0, hca.last_error()
    for bad, word in ((256, "out of range"), (255, "not yet visible")):
        idx = ok.copy()
        idx[0, 9] = bad
        pos = [1000]
        s.check(s.call(pos, idx=idx), pos, idx=idx)
        assert hca.lib.hca_check_device() == -5 and word in hca.last_error()
    table = s.k.table.clone()
    table[0, 1] = -1
    s.k.handle = hca.KvCache("fp4", 512, 64, **s.k.t, block_table=table.cuda())
    idx = np.concatenate([ok[:, :32], np.arange(64, 96)[None]], 1)
    pos = [1023]
    got = s.call(pos, idx=np.concatenate([idx, ok[:, 32:]], 1))
    assert hca.lib.hca_check_device() == -5 and "block-table" in hca.last_error()
    s.check(got, pos, idx=idx)


def test_pool_longer_than_32_bits_of_bytes():
    """Entries at the far end of a pool of 20 M rows (4.5 GB of codes): appended there, attended from there."""
    import long_context_attention_compress_b200 as hca
    n_blocks, rpb, N, H = 625_000, 32, 300, 16
    t = {"codes": torch.empty((n_blocks, rpb, 224), dtype=torch.uint8, device="cuda"),
         "scales": torch.empty((n_blocks, rpb, 16), dtype=torch.uint8, device="cuda"),
         "rope": torch.empty((n_blocks, rpb, 64), dtype=torch.bfloat16, device="cuda")}
    per = -(-N // rpb)
    table = torch.arange(n_blocks - 2 * per, n_blocks, dtype=torch.int32, device="cuda").reshape(2, per)
    k = hca.KvCache("fp4", 512, 64, **t, block_table=table)
    g = torch.Generator().manual_seed(3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    hca.kv_cache_append(torch.randn(2 * N, 512, generator=g).cuda(), k, i32([0, 0]), row_start=i32([0, N, 2 * N]))
    back = to64(hca.kv_cache_gather(k, 2, N))
    assert all(np.abs(back[b]).max() > 1 for b in range(2))
    q = torch.randn(2, H, 512, generator=g).bfloat16()
    cfg = make(512, H)
    got = to64(hca.sparse_mqa_attend_fp4(q.cuda(), k, N, i32([1199, 800]), cfg, rate=4))
    for b, n in enumerate((300, 200)):
        check_query(got[b], to64(q[b]), back[b, :n], cfg.scale, what=f"query {b}")


def test_two_streams_at_once():
    """Calls that run side by side on two streams, each with its workspace, give what they give alone."""
    a, b = Setup(N=900, B=4, rpb=32, seed=1), Setup(N=700, H=16, B=2, nq=8, seed=2)
    calls = [lambda: a.call([3599, 3000, 64, 2000]),
             lambda: b.call([1500 + i % 8 for i in range(16)], q_req=[i // 8 for i in range(16)])]
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
