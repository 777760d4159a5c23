"""The waits of the partial call over an E2M1 cache, made to run out on purpose: with a
limit of a few polls (a test hook, nothing faults) its producer copies nothing, every
warp's wait gives up, and the kernel records the timeout and returns; the calls after it
answer as ever."""
import pytest
import torch

from mla_decode_attention_kv_gb300 import api

from test_gpu_fp4 import Fp4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,q_len", [(16, 1), (24, 1), (64, 1), (128, 2)])
@pytest.mark.parametrize("limit", [1, 8])
def test_fp4_wait_timeout_sets_device_error_and_context_survives(H, q_len, limit):
    lib = api._ffi.lib()
    c = Fp4([3000, 100, 0, 900], H, q_len=q_len, shards=1, bs=64, cur=True, seed=40)
    one = Fp4([256], H, q_len=q_len, bs=64, cur=True, seed=41)
    want = c.run(), c.run(workspace=None), one.run()
    torch.cuda.synchronize()
    try:
        lib.mla_debug_set_spin_limit(limit)
        for k in range(3):
            for run in (c.run, lambda: c.run(workspace=None), one.run):
                c.err.zero_()
                one.err.zero_()
                run()
                torch.cuda.synchronize()
                assert c.err.item() + one.err.item() == 2
    finally:
        lib.mla_debug_set_spin_limit(0)
    c.err.zero_()
    one.err.zero_()
    got = c.run(), c.run(workspace=None), one.run()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    c.check(*got[0])
    one.check(*got[2])
