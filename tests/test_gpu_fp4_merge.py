"""The partial call over an E2M1 cache, row by row (tests/fp4_error.py), and the merge of
cut shards: against whole shards, in every output type, and rounded once."""
import numpy as np
import pytest
import torch

from mla_decode_attention_kv_gb300 import api
from oracle import mla_oracle as om

import fp4_error as fe
from gpu_util import f64
from test_gpu_fp4 import CASES, DEV, TDT, Fp4

pytestmark = pytest.mark.gpu


def check_rows(c, o, batch=None):
    """Every row of o [B, q, P, H, 512] within its bound; returns the bounds [B, q, P, H]."""
    torch.cuda.synchronize()
    assert c.err.item() == 0
    qa, qp, go = f64(c.q_abs), f64(c.q_pe), f64(o)
    h, g = (float(torch.finfo(t).eps) / 2 for t in (TDT[c.dtype], o.dtype))
    bounds = np.zeros(go.shape[:-1])
    for b in range(len(c.lens)) if batch is None else batch:
        cur = None if c.kv_cur is None else f64(c.kv_cur[b])
        segs = om.shard_bounds(len(c.hist[b]), c.S, c.bs)
        for i, p, kv, w in fe.parts(qa[b], qp[b], c.hist[b], cur, api.DEFAULT_SCALE, c.S, segs):
            if w is None:
                assert (go[b, i, p] == 0).all()
                continue
            ref = w @ kv[:, :512]
            bounds[b, i, p] = fe.row_bound(w, kv, ref, h, g)
            # (the scores' fp32 sums: 2^-20 of a row's mean latent at these lengths)
            off = fe.rms(go[b, i, p] - ref) - 2.0 ** -20 * np.sqrt((w @ kv[:, :512] ** 2).mean(-1))
            assert (off <= bounds[b, i, p]).all(), (b, i, p, off.max(), bounds[b, i, p].min())
    return bounds


@pytest.mark.parametrize("name", list(CASES))
def test_fp4_rows_are_within_their_bounds(name):
    c = Fp4(seed=len(name), **CASES[name])
    check_rows(c, c.run()[0])


@pytest.mark.parametrize("H", [5, 16, 32, 64, 100])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("part", ["bf16", "fp16", "fp32"])
def test_fp4_cut_shards_rows(H, dtype, part):
    """Long shards cut between CTAs, in each type: rows within their bounds, next to whole
    shards (both errors together), and the LSEs alike."""
    c = Fp4([9000, 700, 4000], H, shards=1, bs=64, cur=True, dtype=dtype, part=part, seed=H, gain=0.5)
    o1, l1 = c.run()
    bound = check_rows(c, o1)
    o2, l2 = c.run(workspace=None)
    check_rows(c, o2)
    assert (fe.rms(f64(o1) - f64(o2)) <= 2 * bound).all()
    assert (l1 - l2).abs().max().item() <= 2.0 ** -18 * (1 + l1.abs().max().item())


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("part", ["bf16", "fp16"])
def test_fp4_rows_are_rounded_once(H, part):
    """16-bit partials are the fp32 ones rounded, for shards that are cut as for whole ones."""
    c = Fp4([9000, 40, 4000], H, shards=1, bs=64, cur=True, seed=30)
    for ws in ("default", None):
        o32, l32 = c.run(part_dtype=torch.float32, workspace=ws)
        o16, l16 = c.run(part_dtype=TDT[part], workspace=ws)
        assert torch.equal(o32.to(TDT[part]), o16) and torch.equal(l32, l16)


def test_fp4_cut_shards_of_several_query_tokens_and_slices():
    c = Fp4([9000, 4000], 64, q_len=3, shards=2, bs=64, cur=True, seed=31, gain=0.5)
    o1, l1 = c.run()
    check_rows(c, o1)
    o2, l2 = c.run(head_slices=8)
    B, q, P, H, D = o1.shape
    assert torch.equal(o1.reshape(B * q, P, 8, H // 8, D).permute(2, 0, 1, 3, 4), o2)
    assert torch.equal(l1.reshape(B * q, P, 8, H // 8).permute(2, 0, 1, 3), l2)
