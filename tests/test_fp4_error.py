"""The row bound that the E2M1 attention is held to (tests/fp4_error.py), on CPU: weights
and outputs rounded as documented stay within it, and mistakes planted in the merge of a
cut shard do not."""
import numpy as np
import pytest
import torch

import fp4_error as fe

T16 = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _round(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).to(T16[dt]).double().numpy()


def _problem(n, H=4, gain=1.0, seed=0):
    r = np.random.default_rng(seed)
    kv = r.standard_normal((n, 576)) * np.exp(0.4 * r.standard_normal(576))
    q = r.standard_normal((1, H, 576)) * gain
    i, p, kv, w = next(iter(fe.parts(q[..., :512], q[..., 512:], kv, None, 1 / np.sqrt(192), 1, [(0, n)])))
    return kv, w


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 2, 65, 900, 9000])
@pytest.mark.parametrize("gain", [0.0, 1.0, 4.0])
def test_documented_roundings_stay_within_the_bound(dt, n, gain):
    kv, w = _problem(n, gain=gain, seed=n)
    h = float(torch.finfo(T16[dt]).eps) / 2
    ref = w @ kv[:, :512]
    for top in (1.0, 0.7, 40.0):              # the reference maximum need not be the row's
        ws = w / w.max(1, keepdims=True) * top
        got = _round((_round(ws, dt) @ kv[:, :512]) / ws.sum(1, keepdims=True), dt)
        # (equal weights round alike: then the error is e o, within g's and h's terms together)
        bound = fe.row_bound(w, kv, ref, h, h if gain else 2 * h)
        assert (fe.rms(got - ref) <= bound).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("mistake", ["left out", "neighbour's rows", "twice"])
def test_mistakes_in_a_merge_pass_the_bound(dt, mistake):
    """A piece of one tile, any of a shard's, shows in some of eight heads' rows."""
    n, cut = 9000, 64
    kv, w = _problem(n, H=8, gain=0.5, seed=3)
    h = float(torch.finfo(T16[dt]).eps) / 2
    ref = w @ kv[:, :512]
    bound = fe.row_bound(w, kv, ref, h, h)
    for a in range(0, n - 2 * cut, cut):
        x = w.copy()
        if mistake == "left out":
            x[:, a:a + cut] = 0
        elif mistake == "twice":
            x[:, a:a + cut] *= 2
        else:
            s0, s1 = w[:, a:a + cut].sum(1, keepdims=True), w[:, a + cut:a + 2 * cut].sum(1, keepdims=True)
            x[:, a:a + cut] = 0
            x[:, a + cut:a + 2 * cut] *= (s0 + s1) / s1
        x /= x.sum(1, keepdims=True)
        assert (fe.rms(x @ kv[:, :512] - ref) > bound).any(), a
