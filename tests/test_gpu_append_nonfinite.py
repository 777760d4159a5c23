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
