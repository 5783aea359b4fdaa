"""The weights of sparse_mqa_attend_fp4 at c = 512: an output is the float64 one but for its own rounding to bf16.

Logits here are exact in f32 (each query has one channel that is not zero, each row's value there has eight bits, the
scale is 1) and the channels compared are positive in every row, so that sum p|row| = |o| and the bounds are tight.
With p the exact weights,
  - a weight is within 2^-15 (two bf16 terms: the first truncated, within 2^-7; the second, the rest, rounded, within
    2^-8 of it) and 2^-18 (f32: the scaled logit and its reference, |s| <= 8 so within 8 * log2(e) * 2^-23 together, and
    the exponential's 2^-22) of p, relative to p: twice that on o, for the numerator and the denominator;
  - f32 sums over U rows: U * 2^-23 of o, twice;
  - the output's rounding: half a step of bf16 at o, 2^(floor(log2 o) - 8).
A weight rounded once to bf16 (2^-8) would miss the bound in every tenth element or so of a few rows' average."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import fill_rows, values
from test_gpu_mqa_fp4 import Setup, make
from parity_util import to64

pytestmark = pytest.mark.gpu
AT = 500  # the channel (one of the rotary ones, bf16) that the logits come from


def setup(H, N, nq=1, B=2, n_win=4, seed=0, rpb=0):
    s = Setup(H=H, B=B, N=N, nq=nq, n_win=n_win, rpb=rpb, seed=seed)
    rng = np.random.default_rng(seed + 1)
    bf = lambda v: torch.tensor(v).bfloat16()  # noqa: E731

    def rows(n):
        y = rng.uniform(0.5, 6.0, size=(n, 512))
        y[:, AT] = rng.uniform(-2.0, 2.0, size=n)
        return bf(y)
    if N:
        fill_rows(s.k, [s.k.row(b, e) for b in range(B) for e in range(N)], to64(rows(B * N)))
    s.ref = values("fp4", s.k.bytes(), {n: s.k.width(n) for n in s.k.t}, 64)
    s.win = rows(B * s.W).view(B, s.W, 512)
    q = np.zeros((B * nq, H, 512))
    q[..., AT] = rng.uniform(-4.0, 4.0, size=(B * nq, H))
    s.q = bf(q)
    s.cfg = make(512, H, n_win)
    s.cfg.scale = 1.0
    return s


def held(got, q, rows, sink=None, what=""):
    o = oracle.mqa_attend(q, rows, 1.0, sink)
    keep = np.arange(512) != AT
    o, got = o[:, keep], got[:, keep]
    bound = 2.0 ** (np.floor(np.log2(o)) - 8) + o * 2 * (2.0 ** -15 + 2.0 ** -18 + len(rows) * 2.0 ** -23)
    err = np.abs(got - o)
    assert (err <= bound).all(), (what, float((err / bound).max()), float(np.mean(err > bound)))


@pytest.mark.parametrize("H,nq", [(64, 1), (100, 1), (16, 5), (1, 40), (64, 3)])
@pytest.mark.parametrize("N", [0, 3, 140])
def test_weights_are_not_rounded(H, nq, N):
    """One query a request, several with columns of their own, several that share a CTA; sinks."""
    s = setup(H, N, nq=nq, seed=H + N)
    pos = np.concatenate([4 * N + 2 + np.arange(nq), 4 * N + 90 + np.arange(nq)])
    req = None if nq == 1 else np.repeat([0, 1], nq)
    for sink in (None, np.linspace(-3.0, 3.0, H)):
        z = None if sink is None else np.float32(sink).astype(np.float64)
        got = to64(s.call(pos, q_req=req, sink=sink))
        for i, t in enumerate(pos):
            held(got[i], to64(s.q[i]), s.rows(i, int(t), int(i if req is None else req[i]), 4, None), z, f"query {i}")


@pytest.mark.parametrize("rpb", [0, 32])
def test_weights_of_selected_entries(rpb):
    s = setup(64, 400, seed=7, rpb=rpb)
    rng = np.random.default_rng(3)
    idx = np.stack([rng.permutation(400)[:5] for _ in range(2)])
    pos = [1599, 1700]
    got = to64(s.call(pos, idx=idx))
    for i, t in enumerate(pos):
        held(got[i], to64(s.q[i]), s.rows(i, t, i, 4, idx), what=f"query {i}")


def test_weights_of_many_rows_unsplit():
    """More queries than the machine has room for: one CTA walks all of a query's rows, tile after tile."""
    s = setup(64, 420, nq=320, B=1, seed=9)
    pos = 1700 + np.arange(320)
    got = to64(s.call(pos, q_req=np.zeros(320, int)))
    for i in (0, 1, 150, 319):
        held(got[i], to64(s.q[i]), s.rows(i, int(pos[i]), 0, 4, None), what=f"query {i}")


@pytest.mark.parametrize("N", [60, 1000])
def test_split_and_unsplit_queries_agree(N):
    """A query alone, whose rows go to many CTAs, and among 320, where one CTA walks them: both within the bounds above, so
    at most a step of bf16 (and twice the f32 bounds) apart, and on few elements."""
    s = setup(64, N, nq=320, B=1, seed=11)
    pos = 4 * N + 3 + np.arange(320)
    many = s.call(pos, q_req=np.zeros(320, int))
    q = s.q
    for i in (0, 319):
        s.q = q[i:i + 1]
        one = s.call([pos[i]], q_req=[0])
        rows = s.rows(0, int(pos[i]), 0, 4, None)
        a, b = to64(one)[0], to64(many)[i]
        held(a, to64(q[i]), rows, what="split")
        held(b, to64(q[i]), rows, what="unsplit")
        keep = np.arange(512) != AT
        assert np.mean(a[:, keep] != b[:, keep]) <= 0.05
