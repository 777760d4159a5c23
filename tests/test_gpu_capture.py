"""Cache operators captured into graphs: as a process's first calls, on branches that
join, and replayed with other graphs between."""
import os
import subprocess
import sys

import pytest
import torch

from mla_decode_attention_kv_gb300 import api

from test_gpu_fp4 import DEV, Fp4

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
from mla_decode_attention_kv_gb300 import api
from test_gpu_fp4 import Fp4
from test_gpu_append import Case
from test_gpu_pages import Pool
c, a, p = Fp4([5000, 300], {H}, shards=1, bs=64, cur=True, seed=1), Case(20, 4, "e2m1"), Pool([40, 33], 2)
par, kid = p.ids([0, 1]), p.ids([2, 3])
src, dst = p.ids([0, 1]), p.ids([5, 6])
copy = torch.zeros_like(p.cache)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q_out, kv_out = a.run()
    o, lse = c.run()
    api.mla_kv_copy_pages(p.cache, copy, src, dst, err_flag=p.err)
    api.mla_kv_free(p.table, p.lens, p.refs, kid, block_size=16, err_flag=p.err)
    api.mla_kv_fork(p.cache, p.table, p.lens, p.refs, par, kid, err_flag=p.err)
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
a.check(q_out, kv_out)
c.check(o, lse)
assert torch.equal(copy[:, 5:7], p.cache[:, :2])
p.host_fork([0, 1], [2, 3])
p.same()
assert p.err.item() == 0 and a.err.item() == 0
print("fine")
"""


@pytest.mark.parametrize("H", [16, 128])
def test_first_calls_of_a_process_are_captured(H):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, H=H)], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_captured_branches_that_join():
    """Two branches write what the attention behind their join reads: one copies the pages,
    the other the queries; the branches' own outputs come from the graph's memory."""
    c = Fp4([3000, 500], 64, shards=2, bs=64, cur=True, seed=2)
    want_o, want_l = [t.clone() for t in c.run()]
    pages, q = c.pages.clone(), c.q_abs.clone()
    n = pages.shape[0]
    ids = torch.randperm(n, device=DEV).int()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            api.mla_kv_copy_pages(pages, c.pages, ids, ids, err_flag=c.err)
        c.q_abs.copy_(q)
        main.wait_stream(side)
        o, lse = c.run()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            lat = api.mla_lse_combine(o, lse)[0]
        main.wait_stream(side)
    first = None
    for _ in range(5):
        c.pages.zero_()
        c.q_abs.zero_()
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(lse, want_l) and c.err.item() == 0
        first = lat.clone() if first is None else first
        assert torch.equal(lat, first)


def test_graphs_of_one_pool_replayed_in_turn_with_eager_calls():
    """Three graphs that share a memory pool, replayed in any order on one stream with
    eager calls between."""
    cs = [Fp4([4000, 100], H, shards=1, bs=64, seed=H) for H in (16, 32, 64)]
    want = [[t.clone() for t in c.run()] for c in cs]
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for c, w in zip(cs, want):
        g = torch.cuda.CUDAGraph()
        o, lse = torch.empty_like(w[0]), torch.empty_like(w[1])
        with torch.cuda.graph(g, pool=pool):
            c.run(o_part=o, lse_part=lse)
        pool = g.pool()
        graphs.append(g)
        outs.append((o, lse))
    for k in (0, 2, 1, 1, 0, 2):
        for t in outs[k]:
            t.zero_()
        graphs[k].replay()
        eager = cs[(k + 1) % 3].run()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(k + 1) % 3]))


def test_captured_calls_on_a_given_stream():
    """stream= inside a capture, another one current: outputs from the graph's memory."""
    c = Fp4([3000, 500], 16, shards=2, bs=64, cur=True, seed=3)
    want_o, want_l = [t.clone() for t in c.run()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for _ in range(3):
            o, lse = c.run(stream=side)
        lat = api.mla_lse_combine(o, lse, stream=side)[0]
        main.wait_stream(side)
        copy = lat.clone()
    for _ in range(3):
        o.zero_()
        copy.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(lse, want_l) and c.err.item() == 0
        assert torch.equal(copy, api.mla_lse_combine(want_o, want_l)[0])
