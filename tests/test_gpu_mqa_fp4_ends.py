"""sparse_mqa_attend_fp4 at the ends of its range: values that are not finite, logits far from zero, positions up to 2^31 - 1,
split and unsplit queries.  Finite outputs are held to the bounds of test_gpu_mqa_fp4."""

import numpy as np
import pytest
import torch

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
