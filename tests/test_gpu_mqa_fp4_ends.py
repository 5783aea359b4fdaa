"""sparse_mqa_attend_fp4 at the ends of its range: values that are not finite, logits far from zero, positions up to 2^31 - 1,
split and unsplit queries.  Finite outputs are held to the bounds of test_gpu_mqa_fp4."""

import numpy as np
import pytest
import torch

from kv_cache_util import fill_rows, values
from parity_util import to64
from test_gpu_mqa_fp4 import Setup, check_query

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
WIDTHS = [(64, 32, 4), (256, 64, 8), (512, 64, 64)]


@pytest.mark.parametrize("c,rope,H", WIDTHS)
def test_nan_query(c, rope, H):
    """A NaN in one head's query: that head's outputs are NaN, the other heads' and queries' as ever."""
    s = Setup(c=c, rope=rope, H=H, N=40, n_win=16, seed=c)
    clean = s.q.clone()
    s.q[0, 1, 3] = NAN
    pos = [170, 120]
    got = to64(s.call(pos))
    assert np.isnan(got[0, 1]).all()
    other = np.arange(H) != 1
    check_query(got[0][other], to64(clean[0])[other], s.rows(0, 170, 0, 4, None), s.cfg.scale)
    check_query(got[1], to64(clean[1]), s.rows(1, 120, 1, 4, None), s.cfg.scale)


@pytest.mark.parametrize("c,rope,H", WIDTHS)
@pytest.mark.parametrize("slots", [[7], [-1] * 20 + [7], [7] * 33, list(range(8)) + [-1] * 30])
def test_nan_row_among_few(c, rope, H, slots):
    """A NaN row as the only selected one, behind empty slots, selected again and again, and among others: NaN throughout."""
    s = Setup(c=c, rope=rope, H=H, B=2, N=40, seed=c, win=False)
    flat = s.k.t["rope"].view(-1, s.k.t["rope"].shape[-1])
    flat[s.k.row(0, 7), 5] = NAN
    idx = np.tile(slots, (2, 1))
    pos = [170, 171]
    got = to64(s.call(pos, idx=idx))
    assert np.isnan(got[0]).all()
    check_query(got[1], to64(s.q[1]), s.rows(1, 171, 1, 4, idx), s.cfg.scale)


@pytest.mark.parametrize("c,rope,H", WIDTHS)
@pytest.mark.parametrize("n", [1, 5, 300])
@pytest.mark.parametrize("size", [1e14, 1e16])
def test_logits_far_below_zero(c, rope, H, n, size):
    """Logits from -1e29 to -1e36: the least of them takes all the weight, and its row comes out as it is."""
    s = Setup(c=c, rope=rope, H=H, B=2, N=n, seed=n, win=False)
    rng = np.random.default_rng(n)
    y = rng.uniform(0.5, 1.0, size=(2, n, c)) * size * (2.0 + np.arange(n) % 7)[None, :, None]
    y[:, n // 2] *= 0.25  # (below a half of any other row, channel by channel)
    rows = to64(torch.tensor(y).bfloat16()).reshape(2 * n, c)
    fill_rows(s.k, [s.k.row(b, e) for b in range(2) for e in range(n)], rows)
    s.ref = values("fp4", s.k.bytes(), {m: s.k.width(m) for m in s.k.t}, rope)
    s.q = -torch.tensor(rng.uniform(0.5, 1.0, size=(2, H, c)) * size).bfloat16()
    got = to64(s.call([4 * n - 1, 4 * n + 1]))
    for b in range(2):
        np.testing.assert_array_equal(got[b], np.broadcast_to(s.ref[s.k.row(b, n // 2)], (H, c)))


@pytest.mark.parametrize("H,nq", [(64, 1), (16, 3)])
@pytest.mark.parametrize("n", [3, 1000])
@pytest.mark.parametrize("size", [1e2, 1e3, 1e4, 1e5, 1e8])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_large_logits(H, nq, n, size, sign):
    """Logits of either sign from 1e5 to 1e17, several tiles and splits, one that takes all the weight; ordinary logits for one
    head among them."""
    s = Setup(H=H, B=2, N=n, nq=nq, seed=n, win=False, rpb=16)
    rng = np.random.default_rng(n)
    y = rng.uniform(0.5, 1.0, size=(2, n, 512)) * size
    y[:, n // 2] *= 0.25
    y[:, n // 3] *= 4.0
    fill_rows(s.k, [s.k.row(b, e) for b in range(2) for e in range(n)], to64(torch.tensor(y).bfloat16()).reshape(2 * n, 512))
    s.ref = values("fp4", s.k.bytes(), {m: s.k.width(m) for m in s.k.t}, 64)
    q = rng.uniform(0.5, 1.0, size=(2 * nq, H, 512)) * size * sign
    q[:, : H // 2] *= -1
    q[:, 5] /= size * size * 512
    s.q = torch.tensor(q).bfloat16()
    pos = np.concatenate([4 * n - 1 + np.arange(nq), 4 * n + 1 + np.arange(nq)])
    got = to64(s.call(pos, q_req=None if nq == 1 else np.repeat([0, 1], nq)))
    for i in range(2 * nq):
        b = i // nq
        rows = s.rows(i, int(pos[i]), b, 4, None)
        logits = s.cfg.scale * (to64(s.q[i]) @ rows.T)
        top = np.sort(logits, 1)
        clear = top[:, -1] - top[:, -2] > 20 + 2.0 ** -14 * np.abs(top).max(1)  # (told apart by f32 sums of 512 products)
        clear[5] = False
        assert clear.sum() >= H // 4
        np.testing.assert_array_equal(got[i][clear], rows[np.argmax(logits, 1)][clear])
        check_query(got[i][5:6], to64(s.q[i])[5:6], rows, s.cfg.scale)


@pytest.mark.parametrize("c,rope,H", WIDTHS)
@pytest.mark.parametrize("n", [1, 3, 200])
@pytest.mark.parametrize("sink", [False, True])
def test_only_rows_of_infinities(c, rope, H, n, sink):
    """Rows whose logits are all -inf (for half of the heads; +inf for the others): no head's output is finite throughout."""
    s = Setup(c=c, rope=rope, H=H, B=2, N=n, seed=n, win=False)
    flat = s.k.t["rope"].view(-1, s.k.t["rope"].shape[-1])
    for e in range(n):
        flat[s.k.row(0, e), 3] = -INF
    q = s.q.abs()
    q[:, ::2] *= -1
    s.q = q
    pos = [4 * n - 1, 4 * n]
    z = np.linspace(-1, 1, H) if sink else None
    got = to64(s.call(pos, sink=z))
    assert (~np.isfinite(got[0])).any(axis=1).all()
    check_query(got[1], to64(s.q[1]), s.rows(1, 4 * n, 1, 4, None), s.cfg.scale, z)


@pytest.mark.parametrize("c,rope,H", WIDTHS + [(512, 64, 16)])
@pytest.mark.parametrize("rate", [1, 4, 1 << 30, 2 ** 31 - 1])
def test_last_positions(c, rope, H, rate):
    """Queries at 2^31 - 1 and just before it: every entry and the whole window, the output rotated back."""
    s = Setup(c=c, rope=rope, H=H, B=2, N=150, nq=2, n_win=32, seed=c)
    pos = np.array([2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1 - 40])
    req = [0, 0, 1, 1]
    s.check(s.call(pos, rate=rate, q_req=req, rotate=True), pos, rate=rate, q_req=req, rotate=True)


@pytest.mark.parametrize("H", [2, 8, 32])
def test_one_query_a_request_is_planned_the_same_named_or_not(H):
    """Queries of different requests have no rows to share: naming the requests changes neither the plan nor a bit."""
    s = Setup(H=H, B=12, N=700, rpb=32, seed=H)
    pos = 2700 + 9 * np.arange(12)
    assert torch.equal(s.call(pos), s.call(pos, q_req=np.arange(12)))
    req = np.random.default_rng(H).permutation(12)
    s.check(s.call(pos, q_req=req), pos, q_req=req)


def test_chunk_of_one_request_of_a_large_cache():
    """A handful of queries of one request beside many idle ones, and through a descriptor of that request alone."""
    import long_context_attention_compress_b200 as hca
    s = Setup(H=16, B=9, N=300, rpb=32, nq=1, W=140, seed=5)
    pos, req = 1100 + np.arange(9), np.full(9, 4)
    s.check(s.call(pos, q_req=req), pos, q_req=req)
    one = hca.KvCache("fp4", 512, 64, **s.k.t, block_table=s.k.table[4:5].contiguous().cuda())
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = hca.sparse_mqa_attend_fp4(s.q.cuda(), one, 300, i32(pos), s.cfg, rate=4, win=s.win[4:5].contiguous().cuda(),
                                    q_req=i32(np.zeros(9)))
    s.check(got, pos, q_req=req)
