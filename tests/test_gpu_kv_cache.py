"""kv_cache_append and kv_cache_gather on the GPU: every form and arrangement
against the oracle's float64 normalisation, rotation and quantisers.

What is compared.  Codes, scales and unrotated bf16 channels: bit for bit (the
kernel rounds as from the float64 value).  Rotated channels: the two float64
angles differ by a few 2^-53 of |angle| <= 2^20, so a value next to a bf16
midpoint may fall on either side: at most one bf16 step, on at most one element
in a thousand.  All other bytes of the arrays: unchanged."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import Cache, fill_rows, stored, values
from parity_util import to64

pytestmark = pytest.mark.gpu

EPS, BASE = 1e-6, 10000.0


def _x(n, c, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n, c)) * 10.0 ** rng.uniform(-3, 3, size=(n, 1))
    if n > 2:
        x[1, : min(c, 64)] = 0.0
        x[2] *= 1e-25
    return torch.tensor(x).to(dtype)


def _ready(x, entries, rate, gamma, rotate, rope):
    y = to64(x)
    if gamma is not None:
        y = oracle.rms_norm(y, gamma.double().cpu().numpy(), EPS)
    if rotate and rope:
        y = oracle.rope(y, (np.asarray(entries, dtype=np.int64) + 1) * rate - 1, rope, BASE)
    return oracle.round_bf16(y) if gamma is not None or (rotate and rope) else y


def _check(cache, before, rows, y, rotated):
    """Rows `rows` hold y's stored form; every other byte is as before."""
    after, want = cache.bytes(), stored(cache.form, y, cache.rope)
    for k, b in want.items():
        got = after[k][rows][:, : b.shape[1]]
        part = rotated and (k == "rope" or cache.form == "bf16")
        if part:
            u, v = got.reshape(-1, 2).copy().view(np.int16), b.reshape(-1, 2).copy().view(np.int16)
            step = np.abs(u.astype(int) - v.astype(int))
            near = (step <= 1) | (np.abs(to64(torch.tensor(u).view(torch.bfloat16)) -
                                         to64(torch.tensor(v).view(torch.bfloat16))) <= 2.0 ** -30)
            assert near.all() and np.mean(step > 0) <= 1e-3, (k, step.max(), np.mean(step > 0))
        else:
            np.testing.assert_array_equal(got, b, err_msg=k)
        rest = np.ones(after[k].shape, bool)
        rest[np.ix_(rows, np.arange(b.shape[1]))] = False
        np.testing.assert_array_equal(after[k][rest], before[k][rest], err_msg=f"{k}: bytes that are not the new rows'")


FORMS = ["bf16", "fp8", "fp4"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c,rope,rpb,spread", [(512, 64, 32, 0), (512, 64, 0, 2), (512, 0, 1, 0), (128, 0, 7, 1),
                                               (64, 0, 3, 0), (320, 128, 0, 0)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_ragged(form, dtype, c, rope, rpb, spread, norm):
    """Ragged rows of several requests (an empty one and one turned off among them), padding before and behind."""
    import long_context_attention_compress_b200 as hca
    counts, first = [5, 0, 33, 1, 4], [0, 7, 11, -1, 3]
    k = Cache(form, c, rope, len(counts), 48, rpb=rpb, spread=spread)
    lead, n = 2, sum(counts)
    x = _x(lead + n + 3, c, dtype, seed=c + rope)
    start = np.concatenate([[0], np.cumsum(counts)]) + lead
    gamma = torch.tensor(np.random.default_rng(1).uniform(0.5, 1.5, c), dtype=torch.float32).cuda() if norm else None
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, torch.tensor(first, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda(), rate=4, gamma=gamma, rotate=norm,
                        norm_eps=EPS, rope_base=BASE)
    src, rows, ent = [], [], []
    for b, m in enumerate(counts):
        for j in range(m):
            if first[b] >= 0:
                src.append(start[b] + j)
                ent.append(first[b] + j)
                rows.append(k.row(b, first[b] + j))
    _check(k, before, rows, _ready(x[src], ent, 4, gamma, norm, rope), norm and rope > 0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gamma_on,rotate", [(True, True), (True, False), (False, True)])
def test_append_decode_far_positions(form, gamma_on, rotate):
    """One row a request, positions up to 2^20 (rate 128), each switch alone."""
    import long_context_attention_compress_b200 as hca
    B, N = 37, 8192
    k = Cache(form, 512, 64, B, N, rpb=1)
    first = np.random.default_rng(3).integers(0, N, B)
    first[0], first[1] = N - 1, 0
    x = _x(B, 512, torch.float32, seed=9)
    gamma = torch.tensor(np.random.default_rng(2).uniform(0.5, 1.5, 512), dtype=torch.float32).cuda() if gamma_on else None
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, torch.tensor(first, dtype=torch.int32).cuda(), rate=128, gamma=gamma,
                        rotate=rotate, norm_eps=EPS, rope_base=BASE)
    _check(k, before, [k.row(b, int(e)) for b, e in enumerate(first)], _ready(x, first, 128, gamma, rotate, 64), rotate)


@pytest.mark.parametrize("form", FORMS)
def test_append_is_the_separate_calls(form):
    """The same bytes as rms_norm_rope and then the quantiser."""
    import long_context_attention_compress_b200 as hca
    from long_context_attention_compress_b200 import workloads as wl
    cfg = hca.make_cfg(wl.PRO)
    n = 777
    x = _x(n, 512, torch.float32, seed=5).cuda()
    gamma = (torch.rand(512, generator=torch.Generator().manual_seed(1)) + 0.5).cuda()
    k = Cache(form, 512, 64, 1, n)
    hca.kv_cache_append(x, k.handle, torch.zeros(1, dtype=torch.int32, device="cuda"),
                        row_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), rate=4, gamma=gamma, rotate=True,
                        norm_eps=cfg.norm_eps, rope_base=cfg.rope_base)
    y = hca.rms_norm_rope(x, gamma, cfg, pos_add=3, pos_step=4)
    if form == "bf16":
        want = {"codes": y}
    elif form == "fp8":
        codes, scales, rope = hca.kv_fp8_quantize(y, cfg)
        want = {"codes": codes, "scales": scales, "rope": rope}
    else:
        codes, scales = hca.mxfp4_quantize(y[:, :448].contiguous())
        want = {"codes": codes, "scales": scales, "rope": y[:, 448:]}
    for name, w in want.items():
        got = k.t[name][0, :, : w.shape[1]]
        assert torch.equal(got.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), name


@pytest.mark.parametrize("form", FORMS)
def test_append_ring_keeps_the_last_rows(form):
    """A ring of 8 rows given 3, 8 and 21 new rows at once, wrapped."""
    import long_context_attention_compress_b200 as hca
    counts, first, W = [3, 8, 21], [6, 16, 1000003], 8
    k = Cache(form, 512, 64, 3, W, ring=True)
    x = _x(sum(counts), 512, torch.bfloat16, seed=2)
    start = np.concatenate([[0], np.cumsum(counts)])
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, torch.tensor(first, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda())
    src, rows = [], []
    for b, m in enumerate(counts):
        for j in range(max(0, m - W), m):
            src.append(start[b] + j)
            rows.append(k.row(b, first[b] + j))
    _check(k, before, rows, to64(x[src]), False)


def test_append_many_rows_runs():
    """More rows than one per warp: runs that cross request borders, empty requests in a row."""
    import long_context_attention_compress_b200 as hca
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 900, 41)
    counts[5:9] = 0
    k = Cache("fp4", 128, 0, 41, 1000, rpb=32)
    first = rng.integers(0, 100, 41)
    n = int(counts.sum())
    x = _x(n, 128, torch.bfloat16, seed=4)
    start = np.concatenate([[0], np.cumsum(counts)])
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, torch.tensor(first, dtype=torch.int32).cuda(),
                        row_start=torch.tensor(start, dtype=torch.int32).cuda(), rate=4)
    rows = [k.row(b, int(first[b]) + j) for b in range(41) for j in range(counts[b])]
    _check(k, before, rows, to64(x), False)


def test_rows_without_a_place_are_left_out():
    """No room behind the last entry, a block of -1, a block past the pool: nothing is written there, zeros come back,
    and the opt-in check reports it."""
    import long_context_attention_compress_b200 as hca
    k = Cache("fp4", 512, 64, 3, 64, rpb=16)
    table = k.table.clone()
    table[1, 0], table[2, 0] = -1, k.t["codes"].shape[0]
    h = hca.KvCache("fp4", 512, 64, **k.t, block_table=table.cuda())
    before = k.bytes()
    x = _x(6, 512, torch.float32, seed=1).cuda()
    first = torch.tensor([63, 3, 15], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    hca.kv_cache_append(x, h, first, row_start=start)
    # request 0: entry 63 has a row, 64 has none; request 1: none; request 2: entry 16 is in a good block
    _check(k, before, [k.row(0, 63), k.row(2, 16)], to64(x[[0, 5]]), False)
    got = to64(hca.kv_cache_gather(h, 3, 2, first=first))
    assert not got[0, 1].any() and not got[1].any() and not got[2, 0].any() and got[0, 0].any() and got[2, 1].any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("c,rope,rpb,spread", [(512, 64, 32, 0), (512, 0, 0, 1), (128, 0, 5, 0), (320, 128, 1, 2),
                                               (64, 0, 3, 0), (128, 64, 0, 1)])
def test_gather(form, c, rope, rpb, spread):
    """Chosen, consecutive and leading entries; negative and absent ones read as zeros."""
    import long_context_attention_compress_b200 as hca
    B, room = 3, 70
    k = Cache(form, c, rope, B, room, rpb=rpb, spread=spread)
    y = to64(_x(B * room, c, torch.bfloat16, seed=6))
    rows = [k.row(b, e) for b in range(B) for e in range(room)]
    fill_rows(k, rows, y)
    ref = values(form, k.bytes(), {n: k.width(n) for n in k.t}, rope)
    rng = np.random.default_rng(2)
    idx = rng.integers(-2, room, (B, 131))
    idx[0, 3] = 1 << 30
    first = [0, -1, room - 4]

    def want(b, e):
        ok = 0 <= e < room and first is not None
        return oracle.round_bf16(ref[k.row(b, e)]) if ok else np.zeros(c)
    got = to64(hca.kv_cache_gather(k.handle, B, 131, idx=torch.tensor(idx, dtype=torch.int32).cuda()))
    np.testing.assert_array_equal(got, [[want(b, int(e)) for e in idx[b]] for b in range(B)])
    # (a paged cache has room up to the end of its last block; those rows hold the fill)
    m = 4 if rpb else 9
    got = to64(hca.kv_cache_gather(k.handle, B, m, first=torch.tensor(first, dtype=torch.int32).cuda()))
    np.testing.assert_array_equal(got, [[want(b, first[b] + j) if first[b] >= 0 else np.zeros(c) for j in range(m)]
                                        for b in range(B)])
    got = to64(hca.kv_cache_gather(k.handle, B, room))
    np.testing.assert_array_equal(got, [[want(b, j) for j in range(room)] for b in range(B)])


def test_every_fp4_code_and_scale():
    """All 16 codes under every scale byte below 255: exact in bf16, subnormal results included."""
    import long_context_attention_compress_b200 as hca
    k = Cache("fp4", 32, 0, 1, 255)
    codes = np.tile(np.arange(16), 2)[None].repeat(255, 0)
    k.t["codes"][0] = torch.tensor(oracle.mxfp4_pack(codes)).cuda()
    k.t["scales"][0, :, 0] = torch.arange(255, dtype=torch.uint8).cuda()
    got = to64(hca.kv_cache_gather(k.handle, 1, 255))[0]
    want = oracle.mxfp4_dequantize(codes, np.arange(255, dtype=np.uint8)[:, None])
    big = np.abs(want) >= 2.0 ** 128  # 4 and 6 times 2^126, 2 .. 6 times 2^127: past bf16
    np.testing.assert_array_equal(got[~big], want[~big])
    assert np.isinf(got[big]).all()


def test_sequence_longer_than_32_bits_of_elements():
    """Rows whose element offsets pass 2^31: a flat cache of 4.4 M rows of 512 bf16 channels."""
    import long_context_attention_compress_b200 as hca
    n = 4_400_000
    codes = torch.zeros(1, n, 512, dtype=torch.bfloat16, device="cuda")
    h = hca.KvCache("bf16", 512, 64, codes)
    x = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    hca.kv_cache_append(x, h, torch.tensor([n - 3], dtype=torch.int32, device="cuda"),
                        row_start=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert torch.equal(codes[0, -3:], x) and not codes[0, -4].any() and not codes[0, 0].any()
    assert torch.equal(hca.kv_cache_gather(h, 1, 2, idx=torch.tensor([[n - 1, n - 2]], dtype=torch.int32,
                                                                     device="cuda"))[0], x[[2, 1]])


def test_other_stream_and_graph():
    """Given another stream, and captured and replayed with new contents of the same tensors."""
    import long_context_attention_compress_b200 as hca
    k = Cache("fp4", 512, 64, 4, 32, rpb=8)
    x = torch.randn(4, 512, device="cuda")
    first = torch.zeros(4, dtype=torch.int32, device="cuda")
    gamma = torch.rand(512, device="cuda") + 0.5
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    hca.kv_cache_append(x, k.handle, first, rate=4, gamma=gamma, rotate=True, stream=st)
    out = torch.empty(4, 1, 512, dtype=torch.bfloat16, device="cuda")
    hca.kv_cache_gather(k.handle, 4, 1, first=first, out=out, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    a = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hca.kv_cache_append(x, k.handle, first, rate=4, gamma=gamma, rotate=True)
        hca.kv_cache_gather(k.handle, 4, 1, first=first, out=out)
    out.zero_()
    g.replay()
    assert torch.equal(out, a)
    first.fill_(31)
    x.normal_()
    g.replay()
    b = out.clone()
    hca.kv_cache_append(x, k.handle, first, rate=4, gamma=gamma, rotate=True)
    assert torch.equal(hca.kv_cache_gather(k.handle, 4, 1, first=first), b) and not torch.equal(a, b)


def test_debug_check_reports_rows_without_a_place(monkeypatch):
    import long_context_attention_compress_b200 as hca
    k = Cache("bf16", 64, 0, 2, 8)
    x = torch.randn(2, 64, device="cuda")
    assert hca.lib.hca_check_device() == 0
    monkeypatch.setenv("HCA_DEBUG", "1")
    hca.kv_cache_append(x, k.handle, torch.tensor([7, -1], dtype=torch.int32, device="cuda"))
    assert hca.lib.hca_check_device() == 0
    hca.kv_cache_append(x, k.handle, torch.tensor([7, 8], dtype=torch.int32, device="cuda"))
    assert hca.lib.hca_check_device() == -5 and "no place" in hca.last_error()
    assert hca.lib.hca_check_device() == 0


def test_values_that_are_not_finite():
    """bf16 and FP8 keep a NaN; an infinity stays in bf16 and makes its group of 64 channels NaN in FP8; other groups and
    rows are untouched.  FP4 gives finite values of the group's largest magnitude there."""
    import long_context_attention_compress_b200 as hca
    for form in ("bf16", "fp8", "fp4"):
        g = torch.Generator().manual_seed(5)
        x = torch.randn(6, 512, generator=g)
        good = x.clone()
        x[0, 5], x[1, 70], x[2, 511], x[3, 500] = float("nan"), float("inf"), float("nan"), float("-inf")
        out = []
        for rows in (x, good):
            k = Cache(form, 512, 64, 1, 6)
            hca.kv_cache_append(rows.cuda(), k.handle, torch.zeros(1, dtype=torch.int32).cuda(),
                                row_start=torch.tensor([0, 6], dtype=torch.int32).cuda())
            out.append(hca.kv_cache_gather(k.handle, 1, 6)[0].float().cpu())
        y, z = out
        same = torch.ones(6, 512, dtype=torch.bool)
        n = {"bf16": 1, "fp8": 64, "fp4": 32}[form]
        same[0, 5 // n * n:5 // n * n + n] = False
        same[1, 70 // n * n:70 // n * n + n] = False
        same[2, 511] = same[3, 500] = False
        assert torch.equal(y[same], z[same])
        assert torch.isnan(y[2, 511]) and y[3, 500] == float("-inf")  # rotary channels are bf16
        if form == "bf16":
            assert torch.isnan(y[0, 5]) and y[1, 70] == float("inf")
        elif form == "fp8":
            assert torch.isnan(y[0, 5]) and torch.isnan(y[1, 64:128]).all()
            assert torch.isfinite(y[0, 6:]).all()
        else:
            assert torch.isfinite(y[0, :448]).all() and torch.isfinite(y[1, :64]).all()


def test_output_on_another_stream_takes_no_memory_in_use():
    """A call given another stream makes its output there: a block that the current stream has freed, but still reads,
    is not written over."""
    import long_context_attention_compress_b200 as hca
    k = Cache("bf16", 512, 0, 4, 64)
    for _ in range(2):
        x = torch.full((4, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        y = torch.empty_like(x)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # (some ten milliseconds)
        y.copy_(x)
        del x
        out = hca.kv_cache_gather(k.handle, 4, 64, stream=st)
        torch.cuda.synchronize()
        assert (y == 7).all()
        assert torch.equal(out, hca.kv_cache_gather(k.handle, 4, 64))
