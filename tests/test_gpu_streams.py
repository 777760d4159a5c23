"""Calls on another stream than the current one: whose memory their outputs are.

Each test keeps one of the two streams busy (a kernel that spins for some
milliseconds), so that what is ordered wrongly shows."""
import pytest
import torch

from mla_decode_attention_kv_gb300 import api, inputs

from gpu_util import DeviceProblem
from test_gpu_append import Case
from test_gpu_fp4 import Fp4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 30_000_000          # clock ticks: some 15 ms


def _append(kind):
    def make(seed):
        c = Case(40, 8, kind, seed=seed)
        return lambda **kw: c.run(**kw)
    return make


def _fp4(seed):
    c = Fp4([300, 50], 16, cur=True, seed=seed)
    return lambda **kw: c.run(**kw)


def _problem(**over):
    def make(seed):
        dp = DeviceProblem(inputs.make_problem(inputs.DecodeConfig(
            name="s", batch=2, heads=16, q_len=1, num_shards=2, block_size=32, ragged=(1, 200), current=True, seed=seed,
            **over)))
        return dp
    return make


def _partial(seed):
    return _problem()(seed).partial


def _step(seed):
    dp = _problem()(seed)
    return lambda **kw: (dp.step(**kw),)


def _gather(seed):
    dp = _problem()(seed)
    return lambda **kw: (api.mla_gather_kv(dp.cache, dp.table, dp.lens, 200, **kw),)


def _combine(seed):
    dp = _problem()(seed)
    o, lse = dp.partial()
    torch.cuda.synchronize()
    return lambda **kw: api.mla_lse_combine(o, lse, **kw)


CALLS = {"append": _append("e2m1"), "append 16-bit": _append("model"), "fp4": _fp4, "partial": _partial, "step": _step,
         "gather": _gather, "combine": _combine}


def _blocks_like(outs):
    return [torch.empty_like(t) for t in outs]


def _empty_pools():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_are_not_blocks_that_the_current_stream_still_writes(name):
    call, side = CALLS[name](1), torch.cuda.Stream()
    want = [t.clone() for t in call()]
    with torch.cuda.stream(side):
        call()                                   # (the side stream's workspace is there)
    _empty_pools()
    blocks = _blocks_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in blocks:
        t.view(torch.uint8).fill_(0x55)          # still to come on the current stream
    blocks.clear()
    del t
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", list(CALLS))
def test_dropped_outputs_do_not_go_to_the_current_stream_early(name):
    call, side = CALLS[name](2), torch.cuda.Stream()
    want = [t.clone() for t in call(stream=side)]
    _empty_pools()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    call(stream=side)                            # dropped while the side stream has not begun
    blocks = [t.view(torch.uint8).fill_(0x55) for t in _blocks_like(want)]
    torch.cuda.synchronize()
    assert all((t == 0x55).all() for t in blocks)


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_read_on_the_current_stream_stay_until_it_is_done(name):
    call, other, side = CALLS[name](3), CALLS[name](4), torch.cuda.Stream()
    want = [t.clone() for t in call()]
    other(stream=side)
    _empty_pools()
    outs = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in outs]           # still to come
    del outs
    other(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_two_streams_at_once_every_call():
    """The calls of two streams in turn, every one's outputs kept and looked at."""
    cs = [Fp4([5000, 300], 16, shards=1, seed=18), Fp4([4000], 128, shards=2, seed=19)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(6):
        for c, s in zip(cs, streams):
            outs.append((c, c.run(stream=s)))
    torch.cuda.synchronize()
    first = {}
    for c, o in outs:
        if id(c) not in first:
            c.check(*o)
            first[id(c)] = o
        assert all(torch.equal(a, b) for a, b in zip(o, first[id(c)]))


def test_dcp_step_on_another_stream(tmp_path):
    """The sharded step with its exchange on the given stream, over E2M1 pages, a group of
    one rank: the same as the step on the current stream, which is busy meanwhile."""
    import torch.distributed as dist

    from mla_decode_attention_kv_gb300 import dcp
    c = Fp4([300, 50], 16, cur=True, seed=5)
    W = torch.randn(16, 512, 128, device=DEV).to(torch.bfloat16)
    dist.init_process_group("nccl", init_method=f"file://{tmp_path}/rendezvous", rank=0, world_size=1,
                            device_id=torch.device(DEV))
    try:
        def step(**kw):
            return dcp.dcp_decode_step(c.q_abs, c.q_pe, c.pages, c.gtable, c.glens, W, 2, kv_cur=c.kv_cur,
                                       kv_scale=c.kv_scale, err_flag=c.err, **kw)

        want = step()
        o, lse = c.run()
        lat, l2 = api.mla_lse_combine(o, lse)
        torch.cuda.synchronize()
        assert torch.equal(want[1], lat) and torch.equal(want[2], l2)
        assert torch.equal(want[0], api.mla_vup(lat, W))
        side = torch.cuda.Stream()
        step(stream=side)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        got = step(stream=side)
        side.synchronize()                       # (the current stream is still busy)
        with torch.cuda.stream(side):
            copies = [t.clone() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
    finally:
        dist.destroy_process_group()


def test_vup_behind_the_partials_sees_weights_written_before_them():
    """W_UV written by a grid that lets the next one start early, then the partials over
    E2M1 pages and the V-up, which reads W_UV ahead of its wait for the partials: the same
    as with a wait after every call."""
    c = Fp4([300, 50], 16, cur=True, seed=6)
    g = torch.Generator(device=DEV).manual_seed(3)
    Ws = [torch.randn(16, 512, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(6)]
    ids = torch.arange(16, dtype=torch.int32, device=DEV)

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        W, outs = torch.zeros_like(Ws[0]), []
        torch.cuda.synchronize()
        for k in range(60):
            api.mla_kv_copy_pages(Ws[k % 6], W, ids, ids, err_flag=c.err)
            sync()
            o, lse = c.run()
            sync()
            outs.append(api.mla_lse_combine_vup(o, lse, W, err_flag=c.err))
            sync()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        return outs

    assert all(torch.equal(a, b) for a, b in zip(run(False), run(True)))
