"""mla_kv_append over drawn sizes and layouts: queries heads first or tokens first, rows of
wider projections, outputs given, padded and long batches."""
import random

import pytest
import torch

from mla_decode_attention_kv_gb300 import api
from mla_decode_attention_kv_gb300._ffi import MlaError

from test_gpu_append import BF, DEV, HF, Case

pytestmark = pytest.mark.gpu


def _place(x, how, r):
    """x [T, H, 64] as a view with other strides and the same values."""
    T, H, _ = x.shape
    if how == "heads first":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    pad = 8 * r.randint(0, 5)
    if how == "wider":
        buf = torch.full((T, H, 64 + pad + 8), 7.0, dtype=x.dtype, device=x.device)
        buf[:, :, pad:pad + 64] = x
        return buf[:, :, pad:pad + 64]
    if how == "shared":                       # one head's queries for all heads
        return x[:, :1].expand(T, H, 64)
    return x


@pytest.mark.parametrize("seed", range(40))
def test_drawn_layouts(seed):
    r = random.Random(seed)
    T, H = r.choice([1, 2, 3, 31, 64, r.randint(1, 400)]), r.choice([1, 2, 15, 16, 17, 33, 128])
    kind, dt = r.choice(["model", "e4m3", "e2m1"]), r.choice([BF, HF])
    c = Case(T, H, kind, dt, axes=r.choice([1, 2, 3]), interleaved=r.random() < .5, bs=r.choice([16, 32, 64, 128, 256]),
             seed=seed, weight=r.random() < .8, pad=r.random() < .5, strided=r.random() < .5)
    how = r.choice(["as is", "heads first", "wider", "shared"])
    c.q_pe = _place(c.q_pe.contiguous(), how, r)
    given = r.choice(["none", "plain", "heads first", "wider"])
    if given == "none":
        q_out, kv_out = c.run()
    else:
        want = _place(torch.full((T, H, 64), 9.0, dtype=dt, device=DEV), given, r)
        kv_dt = torch.uint8 if kind == "e4m3" else dt
        kv = torch.empty(T, 576, dtype=kv_dt, device=DEV)
        q_out, kv_out = c.run(q_out=want, kv_out=kv)
        assert q_out.data_ptr() == want.data_ptr() and kv_out.data_ptr() == kv.data_ptr()
        if given == "wider" and T * H > 1:
            rest = torch.as_strided(want, (T * H - 1,), (want.stride(1),), want.storage_offset() + 64)
            assert (rest == 7).all()          # between the rows: left alone
    torch.cuda.synchronize()
    assert c.err.item() == 0
    c.check(q_out, kv_out)


@pytest.mark.parametrize("kind", ["model", "e4m3", "e2m1"])
def test_a_long_batch_and_one_that_is_all_padding(kind):
    c = Case(40000, 1, kind, bs=64, seed=50)
    c.check(*c.run())
    p = Case(33, 5, kind, bs=64, seed=51)
    p.slots.fill_(-1)
    before = p.cache.clone()
    p.check(*p.run())
    assert torch.equal(p.cache, before) and p.err.item() == 0


def test_calls_without_tokens():
    c = Case(0, 3, "e2m1", pad=False)
    q_out, kv_out = c.run()
    assert q_out.shape == (0, 3, 64) and kv_out.shape == (0, 576) and (c.cache == 3).all()


def test_outputs_whose_rows_overlap_are_refused():
    c = Case(8, 4, "model")
    for bad in (torch.empty(8, 1, 64, dtype=BF, device=DEV).expand(8, 4, 64),
                torch.empty(1, 4, 64, dtype=BF, device=DEV).expand(8, 4, 64),
                torch.empty(8 * 4 * 64, dtype=BF, device=DEV).as_strided((8, 4, 64), (64, 64, 1))):
        with pytest.raises(MlaError):
            c.run(q_out=bad)
    with pytest.raises(MlaError):             # q_pe's own memory at other strides
        c.q_pe = torch.randn(8, 4, 64, dtype=BF, device=DEV)
        c.run(q_out=c.q_pe.as_strided((8, 4, 64), (64, 512, 1)))
    want, kv = c.run()
    got, _ = c.run(q_out=c.q_pe)
    assert torch.equal(got, want)
