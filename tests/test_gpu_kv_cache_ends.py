"""kv_cache_append and kv_cache_gather at the ends of their range: magnitudes near f32's limits, and launches large enough
that a warp or a block walks several rows.  Compared as in test_gpu_kv_cache: codes, scales and unrotated bf16 channels bit
for bit with the oracle's float64 values, rotated channels within a bf16 step."""

import numpy as np
import pytest
import torch

import oracle
from kv_cache_util import Cache, values
from test_gpu_kv_cache import BASE, FORMS, _check, _ready

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _normed(x, entries, rate, gamma, eps, rope):
    y = oracle.rms_norm(x.double().numpy(), gamma.double().numpy(), eps)
    return oracle.round_bf16(oracle.rope(y, (np.asarray(entries, dtype=np.int64) + 1) * rate - 1, rope, BASE))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("gammas", ["up to 2", "far apart"])
def test_append_normalises_any_magnitude(form, dtype, eps, gammas):
    """Rows from f32's subnormals to its largest values, with and without an eps that outweighs them, single channels far
    below their row's: products that pass f32's range on the way to an ordinary value."""
    import long_context_attention_compress_b200 as hca
    rng = np.random.default_rng(1)
    scales = [3.3e38, 2.6e38, 1e38, 3e37, 1e30, 1e13, 1.0, 1e-13, 1e-30, 1e-37, 1e-38, 1e-40]
    if dtype is torch.float32:
        scales.append(1e-43)  # (below bf16's least)
    x = rng.uniform(0.5, 1.0, size=(2 * len(scales), 512)) * rng.choice([-1.0, 1.0], size=(2 * len(scales), 512))
    x *= np.repeat(scales, 2)[:, None]
    x[1::2, ::5] *= 10.0 ** rng.uniform(-45, 0, size=x[1::2, ::5].shape)  # (some become zeros)
    x = torch.tensor(x).to(dtype)
    assert torch.isfinite(x).all()
    gamma = torch.tensor(rng.uniform(0.5, 2.0, 512), dtype=torch.float32)
    if gammas == "far apart":
        gamma[::7] *= 2.0 ** 70
        gamma[3::7] *= 2.0 ** -70
        gamma[5::49] = 0.0
    n = len(x)
    k = Cache(form, 512, 64, 1, n, rpb=8)
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, _i32([0]), row_start=_i32([0, n]), rate=4, gamma=gamma.cuda(), rotate=True,
                        norm_eps=eps, rope_base=BASE)
    _check(k, before, [k.row(0, e) for e in range(n)], _normed(x, np.arange(n), 4, gamma, float(np.float32(eps)), 64), True)


def _tiny_rows():
    """Rows whose largest magnitude is a few of f32's least steps: amax / 448 is 0 in f32 up to 224 of them."""
    rng = np.random.default_rng(2)
    steps = rng.integers(-3, 4, size=(6, 512)) * np.array([1, 10, 60, 74, 100, 1000])[:, None]
    steps[0, :64] = 0
    return torch.tensor(steps * 2.0 ** -149).float()


def _tiny_form(x):
    """FP8 form of such rows: under a scale of 0 a value that is not 0 takes the largest code of its sign."""
    y = x[:, :448].double().numpy().reshape(len(x), 7, 64)
    amax = np.abs(y).max(-1)
    scale = np.where(amax > 0, amax / 448.0, 1.0).astype(np.float32)
    q = np.where(scale[..., None] == 0, np.sign(y) * 448.0, y / np.where(scale == 0, 1, scale).astype(np.float64)[..., None])
    codes = torch.tensor(oracle.round_e4m3(q)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(len(x), 448), torch.tensor(scale)


def test_fp8_groups_whose_scale_rounds_to_zero():
    """Rows converted as they are: the bytes are the form's, and the rows read back as zeros, not as 0 / 0."""
    import long_context_attention_compress_b200 as hca
    x = _tiny_rows()
    k = Cache("fp8", 512, 64, 1, 6)
    hca.kv_cache_append(x.cuda(), k.handle, _i32([0]), row_start=_i32([0, 6]))
    codes, scales = _tiny_form(x)
    assert torch.equal(k.t["scales"][0].cpu(), scales)
    got = k.t["codes"][0].cpu()
    assert torch.equal(torch.where(got == 128, 0, got), torch.where(codes == 128, 0, codes))  # (a zero of either sign)
    back = hca.kv_cache_gather(k.handle, 1, 6)[0].float().cpu()
    assert (back[:4, :448] == 0).all()  # (up to 222 steps)
    assert torch.isfinite(back).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_fp8_form_is_one_for_both_calls(dtype):
    """kv_fp8_quantize writes what kv_cache_append does also for groups whose scale rounds to 0, for NaN (kept) and for
    infinities (whose group reads as NaN); no value reaches its neighbours' codes."""
    import long_context_attention_compress_b200 as hca
    from long_context_attention_compress_b200 import workloads as wl
    at = [(6, 5), (8, 2), (8, 3), (8, 4), (7, 70), (9, 200)]
    x = torch.cat([_tiny_rows(), torch.randn(4, 512, generator=torch.Generator().manual_seed(4))]).to(dtype)
    for r, c in at:
        x[r, c] = 0.01  # (not its group's largest)
    good = x.clone()
    for (r, c), v in zip(at, [float("nan")] * 4 + [float("inf"), -float("inf")]):
        x[r, c] = v
    k = Cache("fp8", 512, 64, 1, 10)
    hca.kv_cache_append(x.cuda(), k.handle, _i32([0]), row_start=_i32([0, 10]))
    cfg = hca.make_cfg(wl.PRO)
    got = dict(zip(("codes", "scales", "rope"), hca.kv_fp8_quantize(x.cuda(), cfg)))
    for name, t in got.items():
        assert torch.equal(k.t[name][0].contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)), name
    codes = got["codes"].cpu()
    assert all(int(codes[r, c]) & 127 == 127 for r, c in at)
    want = hca.kv_fp8_quantize(good.cuda(), cfg)[0].cpu()
    same = torch.ones_like(codes, dtype=torch.bool)
    for r, c in at[:4]:
        same[r, c] = False
    same[7, 64:128] = same[9, 192:256] = False
    assert torch.equal(codes[same], want[same])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,gamma_on,rotate", [(torch.float32, True, True), (torch.bfloat16, True, True),
                                                   (torch.float32, True, False), (torch.float32, False, True),
                                                   (torch.bfloat16, False, False)])
def test_append_several_rows_a_warp(form, dtype, gamma_on, rotate):
    """More rows than one a warp (some 3,600 where they are normalised, 5,900 at most): each warp takes a run of them, with
    the ends of requests and empty requests inside."""
    import long_context_attention_compress_b200 as hca
    rng = np.random.default_rng(3)
    counts = rng.integers(1, 9, 2400)
    counts[7::11] = 0
    counts[1200:1204] = [700, 0, 0, 900]
    B, n, lead = len(counts), int(counts.sum()), 3
    assert n > 10_000
    first = rng.integers(0, 20, B)
    first[50::97] = -1
    k = Cache(form, 512, 64, B, 28, rpb=4)  # (19 + 8 entries at most)
    first[1200], first[1203] = -1, 0
    per = k.table.shape[1]
    # (of the two long requests one is turned off and one has blocks of its own behind the others')
    table = torch.cat([k.table, torch.full((B, 240 - per), -1, dtype=torch.int32)], 1)
    t = {name: torch.cat([v, v[:1].expand(240, *v.shape[1:])]).contiguous() for name, v in k.t.items()}
    table[1203] = torch.arange(240, dtype=torch.int32) + k.t["codes"].shape[0]
    k.t, k.table = t, table
    k.handle = hca.KvCache(form, 512, 64, **t, block_table=table.cuda())
    x = torch.tensor(rng.normal(size=(lead + n + 5, 512)) * 10.0 ** rng.uniform(-2, 2, size=(lead + n + 5, 1))).to(dtype)
    start = np.concatenate([[0], np.cumsum(counts)]) + lead
    gamma = torch.tensor(rng.uniform(0.5, 1.5, 512), dtype=torch.float32) if gamma_on else None
    before = k.bytes()
    hca.kv_cache_append(x.cuda(), k.handle, _i32(first), row_start=_i32(start), rate=128,
                        gamma=None if gamma is None else gamma.cuda(), rotate=rotate, norm_eps=1e-6, rope_base=BASE)
    on = [(start[b] + j, first[b] + j, b) for b in range(B) if first[b] >= 0 for j in range(counts[b])]
    src, ent, req = (np.array(v) for v in zip(*on))
    rows = [k.row(int(b), int(e)) for b, e in zip(req, ent)]
    _check(k, before, rows, _ready(x[src], ent, 128, None if gamma is None else gamma.cuda(), rotate, 64), rotate)


def _random_cache(form, c, rope, B, room, rpb, seed):
    """A cache of random codes, scales of ordinary size and random rotary channels."""
    k = Cache(form, c, rope, B, room, rpb=rpb, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if form == "bf16":
        k.t["codes"].normal_(generator=g)
    else:
        k.t["codes"].random_(0, 127, generator=g)  # (FP8: no NaN)
        k.t["codes"] += 128 * torch.randint(0, 2, k.t["codes"].shape, generator=g, device="cuda").to(torch.uint8)
        k.t["scales"].uniform_(0.01, 2.0, generator=g) if form == "fp8" else k.t["scales"].random_(120, 135, generator=g)
        if rope:
            k.t["rope"].normal_(generator=g)
    return k


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("c,rope,n_out,rpb", [(512, 64, 8667, 32), (512, 0, 13001, 0), (128, 0, 40_001, 32), (64, 0, 33_333, 0)])
def test_gather_several_rounds_a_block(form, c, rope, n_out, rpb):
    """More rows than the resident blocks take at once (11,840, and 47,360 of at most 128 channels): chosen, consecutive and
    leading entries, in numbers that end inside a block's round."""
    import long_context_attention_compress_b200 as hca
    B, room = 3, n_out + 10
    k = _random_cache(form, c, rope, B, room, rpb, seed=c + rpb)
    ref = torch.tensor(values(form, k.bytes(), {n: k.width(n) for n in k.t}, rope)).float().bfloat16()
    ref = torch.cat([ref, torch.zeros(1, c, dtype=torch.bfloat16)])  # (the last: no row)
    at = np.array([[k.row(b, e) for e in range(room)] for b in range(B)])
    rng = np.random.default_rng(1)
    idx = rng.integers(-3, room, (B, n_out))
    rows = np.where(idx >= 0, np.take_along_axis(at, np.maximum(idx, 0), 1), -1)
    got = hca.kv_cache_gather(k.handle, B, n_out, idx=_i32(idx))
    assert torch.equal(got.cpu(), ref[rows])
    first = [0, 7, -1]
    want = [at[0, :n_out], at[1, 7:7 + n_out], np.full(n_out, -1)]
    assert torch.equal(hca.kv_cache_gather(k.handle, B, n_out, first=_i32(first)).cpu(), ref[np.stack(want)])
    assert torch.equal(hca.kv_cache_gather(k.handle, B, n_out).cpu(), ref[at[:, :n_out]])
