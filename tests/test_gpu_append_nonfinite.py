"""mla_kv_append on infinities, NaN and values near the ends of their type: the same as
its formulas in 64 bits, whatever the cache's format."""
import numpy as np
import pytest
import torch

import cache_util as cu
from gpu_util import f64
from test_gpu_append import BF, DEV, HF, Case

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def check(c, kv_out):
    """The stored row of every token and kv_out against the rows in 64 bits."""
    torch.cuda.synchronize()
    assert c.err.item() == 0
    with np.errstate(all="ignore"):
        rows = c.rows()[0]
        slots = c.slots.cpu().numpy()
        if c.kind == "model":
            flat = c.cache.view(-1, 576)[torch.from_numpy(slots).to(DEV).long()]
            assert torch.equal(flat.view(torch.int16), kv_out.view(torch.int16))
            got, fin = f64(kv_out), np.isfinite(rows)
            big = float(torch.finfo(c.dt).max)
            half = float(torch.finfo(c.dt).eps) / 2
            tiny = float(torch.finfo(c.dt).smallest_normal) * half        # half a subnormal step
            assert np.array_equal(np.isnan(got), np.isnan(rows))
            over = fin & (np.abs(rows) > big * (1 + half / 2))             # past the type: an infinity
            assert np.array_equal(got[np.isinf(rows)], rows[np.isinf(rows)]) and np.isinf(got[over]).all()
            fin &= np.abs(rows) < big
            assert np.all(np.abs(got[fin] - rows[fin]) <= half * np.abs(rows[fin]) * (1 + 2.0 ** -20) + tiny)
            return
        if c.kind == "e4m3":
            want = cu.e4m3_bytes(rows / c.kv_scale)
            got = kv_out.view(torch.uint8).cpu().numpy()
            assert np.array_equal(c.cache.cpu().numpy().reshape(-1, 576)[slots], got)
            nan = np.isnan(rows)
            assert np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
            return
        codes, scales = cu.e2m1_rows(rows, c.kv_scale)
        gc, gs = cu.split_pages(c.cache.cpu().numpy())
        gc, gs = gc.reshape(-1, 288)[slots], gs.reshape(-1, 36)[slots]
        nan = np.isnan(rows.reshape(-1, 36, 16)).any(-1)
        assert np.array_equal(gs[~nan], scales[~nan]) and (gs[nan] == 0x7F).all()
        same = gc.reshape(-1, 36, 8) == codes.reshape(-1, 36, 8)
        assert same[~nan].all()                                            # (a NaN block's codes mean nothing)
        got = f64(kv_out).reshape(-1, 36, 16)
        assert np.isnan(got[nan]).all()
        vals = cu.e2m1_values(codes, scales, c.kv_scale).reshape(-1, 36, 16)
        assert np.all(np.abs(got[~nan] - vals[~nan]) <= 2.0 ** -8 * np.abs(vals[~nan]))


KINDS = pytest.mark.parametrize("kind", ["model", "e4m3", "e2m1"])
SHAPE = pytest.mark.parametrize("interleaved", [True, False])


@KINDS
@SHAPE
@pytest.mark.parametrize("dt", [BF, HF])
def test_keys_with_infinities_and_nan(kind, interleaved, dt):
    """An infinite key value stays one (saturated in 8 and 4 bits); beside an infinity of
    its pair, or under a cosine of 0, it is NaN as the formula is."""
    c = Case(9, 1, kind, dt, interleaved=interleaved, pad=False, seed=2)
    c.positions[0, 8] = 0                                   # cos 1, sin 0: 0 times an infinity
    pair = (4, 5) if interleaved else (4, 36)
    k = c.kv_a[:, 512:]
    k[1, pair[0]], k[2, pair[1]], k[3, pair[0]] = INF, -INF, -INF
    k[4, pair[0]], k[4, pair[1]] = INF, INF
    k[5, pair[0]] = NAN
    k[6, pair[0]], k[6, pair[1]] = INF, NAN
    k[7, :] = INF
    k[8, pair[1]] = INF
    check(c, c.run()[1])


@KINDS
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("dt", [BF, HF])
def test_latents_with_infinities_and_nan(kind, weight, dt):
    """With the norm an infinite latent makes its row zeros (signed) and itself NaN, a NaN
    all of the row NaN; without it they go to the cache as they are."""
    c = Case(7, 1, kind, dt, pad=False, weight=weight, seed=3)
    lat = c.kv_a
    lat[1, 17] = INF
    lat[2, 511] = -INF
    lat[3, 0] = NAN
    lat[4, 5], lat[4, 100] = INF, NAN
    lat[5, 3:40] = 0
    lat[5, 7] = INF
    lat[6, 9], lat[6, 10] = INF, -INF
    check(c, c.run()[1])


@KINDS
@pytest.mark.parametrize("size", [1e15, 1e18, 3e19, 1e25, 1e36, 1e38])
def test_rows_whose_squares_pass_fp32(kind, size):
    """bf16 latents up to the type's end: normalised like any others."""
    c = Case(20, 1, kind, BF, pad=False, seed=4)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.rand(20, 512, generator=g, device=DEV) * 2 - 1
    c.kv_a[:, :512] = (x * size).to(BF)
    c.kv_a[3, 1:] = 1.0                                     # one huge value among small ones
    c.kv_a[4] = 0
    check(c, c.run()[1])


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
@pytest.mark.parametrize("kv_scale", [2.0 ** -99, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60, 2.0 ** 99])
def test_scales_at_the_ends_of_their_range(kind, kv_scale):
    """Rows and weights that such scales are for: values of some kv_scale."""
    c = Case(40, 1, kind, BF, pad=False, seed=6, kv_scale=kv_scale)
    c.weight = (c.weight.float() * min(kv_scale, 2.0 ** 60)).to(BF)
    c.kv_a[20:, :512] = (c.kv_a[20:, :512].float() * 2.0 ** 62).to(BF)
    check(c, c.run()[1])


def test_scale_times_norm_below_the_normal_range():
    """1 / kv_scale times the norm's factor below 2^-126: an E4M3 code taken by that
    product would miss borders.  (c * w stays within fp32, |c| < 6 * 2^38, w < 4 * 2^85.)"""
    c = Case(6000, 1, "e4m3", BF, pad=False, seed=7, kv_scale=2.0 ** 94, bs=64)
    c.weight = (c.weight.float() * 2.0 ** 85).to(BF)
    c.kv_a[:, :512] = (torch.randn(6000, 512, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV)
                       * 2.0 ** 38).clamp(-6 * 2.0 ** 38, 6 * 2.0 ** 38).to(BF)
    check(c, c.run()[1])
