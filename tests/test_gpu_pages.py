"""mla_kv_fork, mla_kv_free and mla_kv_copy_pages against plain Python loops."""
import numpy as np
import pytest
import torch

from mla_decode_attention_kv_gb300 import api
from mla_decode_attention_kv_gb300._ffi import MlaError

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Pool:
    """`live` sequences of the given lengths over shuffled pages, `empty` empty rows."""

    def __init__(self, lens, empty, bs=16, layers=2, width=324, spare=20, dtype=torch.uint8, seed=0, extra_cols=3):
        r = np.random.RandomState(seed)
        self.bs, R = bs, len(lens) + empty
        per = [-(-n // bs) for n in lens]
        blocks = sum(per) + spare
        perm = r.permutation(blocks)
        table = np.full((R, max(per + [1]) + extra_cols), -1, np.int32)
        refs = np.zeros(blocks, np.int32)
        at = 0
        for i, n in enumerate(per):
            table[i, :n] = perm[at:at + n]
            refs[perm[at:at + n]] += 1
            at += n
        self.h = dict(table=table, lens=np.array(list(lens) + [0] * empty, np.int32), refs=refs,
                      cache=r.randint(0, 256, (layers, blocks, bs, width * dtype.itemsize)).astype(np.uint8))
        self.table, self.lens, self.refs = (torch.from_numpy(self.h[k].copy()).to(DEV) for k in ("table", "lens", "refs"))
        self.cache = torch.from_numpy(self.h["cache"].copy()).to(DEV).view(dtype)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def ids(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def fork(self, parents, children, **kw):
        api.mla_kv_fork(self.cache, self.table, self.lens, self.refs, self.ids(parents), self.ids(children),
                        err_flag=self.err, **kw)
        torch.cuda.synchronize()

    def free(self, rows):
        api.mla_kv_free(self.table, self.lens, self.refs, self.ids(rows), block_size=self.bs, err_flag=self.err)
        torch.cuda.synchronize()

    def host_fork(self, parents, children):
        h = self.h
        # the free pages of the call, the lowest first; shared pages are never free
        free = [int(x) for x in np.nonzero(h["refs"] <= 0)[0]]
        for p, c in zip(parents, children):
            L = int(h["lens"][p])
            h["table"][c] = -1
            for j in range(L // self.bs):
                h["table"][c, j] = h["table"][p, j]
                h["refs"][h["table"][p, j]] += 1
            if L % self.bs:
                f, j = free.pop(0), L // self.bs
                h["table"][c, j] = f
                h["refs"][f] = 1
                h["cache"][:, f] = h["cache"][:, h["table"][p, j]]
            h["lens"][c] = L

    def host_free(self, rows):
        h = self.h
        for r in rows:
            for j in range(-(-int(h["lens"][r]) // self.bs)):
                h["refs"][h["table"][r, j]] -= 1
                h["table"][r, j] = -1
            h["lens"][r] = 0

    def same(self):
        for k in ("table", "lens", "refs"):
            assert np.array_equal(getattr(self, k).cpu().numpy(), self.h[k]), k
        assert np.array_equal(self.cache.view(torch.uint8).cpu().numpy(), self.h["cache"]), "cache"


@pytest.mark.parametrize("bs,layers,width,dtype", [(16, 1, 324, torch.uint8), (64, 3, 576, torch.bfloat16),
                                                   (256, 2, 576, torch.uint8), (32, 2, 324, torch.uint8)])
def test_fork_and_free_match_the_host(bs, layers, width, dtype):
    lens = [0, 1, bs - 1, bs, bs + 1, 3 * bs, 5 * bs + 7]
    p = Pool(lens, 9, bs, layers, width, dtype=dtype)
    parents, children = [1, 6, 6, 3, 0, 2, 4, 5], [7, 9, 8, 10, 11, 15, 13, 12]
    p.fork(parents, children)
    p.host_fork(parents, children)
    p.same()
    # a fork of forks, then parents and some children given back
    p.fork([9], [14])
    p.host_fork([9], [14])
    p.same()
    p.free([6, 9, 3, 0])
    p.host_free([6, 9, 3, 0])
    p.same()
    # the freed pages are taken again, the lowest first
    p.fork([8, 8], [9, 6])
    p.host_fork([8, 8], [9, 6])
    p.same()
    assert p.err.item() == 0


def test_free_of_everything_and_of_a_row_twice():
    p = Pool([40, 17, 100], 3)
    p.fork([0, 2], [3, 4])
    p.host_fork([0, 2], [3, 4])
    p.free([0, 0, 4, 3, 1, 2, 5, 4])
    p.host_free([0, 4, 3, 1, 2, 5])
    p.same()
    assert p.err.item() == 0 and not p.refs.any() and (p.table == -1).all()


def test_fork_many_rows_over_a_large_pool():
    """More pairs than the plan's block has threads, and a pool whose free pages
    lie behind many taken ones."""
    r = np.random.RandomState(5)
    lens = list(r.randint(0, 300, 500))
    p = Pool(lens, 1500, 16, 1, 324, spare=1600, seed=5)
    parents = [int(x) for x in r.randint(0, 500, 1500)]
    children = [int(x) for x in 500 + r.permutation(1500)]
    p.fork(parents, children)
    p.host_fork(parents, children)
    p.same()
    assert p.err.item() == 0


@pytest.mark.parametrize("parents,children,code", [
    ([0, 1], [3, 3], 6),        # into one row twice
    ([0, 1], [3, 1], 6),        # into a row that is taken
    ([0, 3], [3, 4], 6),        # a parent that is a child
    ([0, 9], [3, 4], 6),        # no such row
    ([-1], [3], 6),
    ([0], [9], 6),
    ([0, 1, 2], [3, 4, 5], 7),  # three copies, two free pages
])
def test_fork_errors_change_nothing(parents, children, code):
    p = Pool([20, 30, 40], 5, spare=2)
    p.fork(parents, children)
    assert p.err.item() == code
    p.same()


def test_fork_of_a_bad_length_changes_nothing():
    p = Pool([20, 30], 2)
    p.lens[1] = p.h["lens"][1] = 10 ** 6
    p.fork([0, 1], [2, 3])
    assert p.err.item() == 3
    p.same()


def test_bad_pages_are_recorded():
    p = Pool([40, 17], 2)
    p.table[0, 1] = 10 ** 6
    p.fork([0], [2])
    assert p.err.item() == 1
    p.err.zero_()
    p.free([0])
    assert p.err.item() == 1
    q = Pool([40], 1)
    q.refs.zero_()
    q.free([0])
    assert q.err.item() == 8 and not q.refs.any()
    q.err.zero_()
    q.free([7])
    assert q.err.item() == 6


def test_copy_pages():
    r = np.random.RandomState(3)
    for layers, n, width, dtype in ((1, 1, 324, torch.uint8), (3, 40, 576, torch.bfloat16), (2, 7, 576, torch.uint8)):
        mk = lambda k: torch.from_numpy(r.randint(0, 256, (layers, k, 32, width * dtype.itemsize)).astype(np.uint8)).to(DEV)  # noqa: E731
        src, dst = mk(50), mk(45)
        a, b = r.permutation(50)[:n], r.permutation(45)[:n]
        want = dst.clone()
        want[:, b] = src[:, a]
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = api.mla_kv_copy_pages(src.view(dtype), dst.view(dtype), torch.tensor(a, dtype=torch.int32, device=DEV),
                                    torch.tensor(b, dtype=torch.int32, device=DEV), err_flag=err)
        assert torch.equal(got.view(torch.uint8), want) and err.item() == 0


def test_copy_within_a_pool_of_strided_layers_and_bad_ids():
    base = torch.randint(0, 256, (4, 30, 16, 324), dtype=torch.uint8, device=DEV)
    pool = base[::2]                              # every second layer
    want = base.clone()
    want[::2, 29] = want[::2, 0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    api.mla_kv_copy_pages(pool, pool, ids(0), ids(29), err_flag=err)
    assert torch.equal(base, want) and err.item() == 0
    want[::2, 3] = want[::2, 2]
    api.mla_kv_copy_pages(pool, pool, ids(30, 2, 5, -1), ids(1, 3, 30, 4), err_flag=err)
    assert torch.equal(base, want) and err.item() == 1


def test_fork_in_a_graph():
    p = Pool([40, 33], 2, spare=8)
    par, kid = p.ids([0, 1]), p.ids([2, 3])
    ws = torch.empty(64, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mla_kv_free(p.table, p.lens, p.refs, kid, block_size=16, err_flag=p.err)
        api.mla_kv_fork(p.cache, p.table, p.lens, p.refs, par, kid, workspace=ws, err_flag=p.err)
    p.host_fork([0, 1], [2, 3])
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        p.same()
    assert p.err.item() == 0


def test_fork_into_strided_layers_and_back_to_back():
    """Layers that are views of a larger tensor, and three forks in a row on one stream
    (each starts while the one before ends)."""
    p = Pool([40, 33, 100], 6, layers=3)
    base = torch.zeros(6, *p.cache.shape[1:], dtype=torch.uint8, device=DEV)
    base[::2] = p.cache
    p.cache = base[::2]
    for a, b in (([0, 1], [3, 4]), ([3, 2], [5, 6]), ([6, 4], [7, 8])):
        api.mla_kv_fork(p.cache, p.table, p.lens, p.refs, p.ids(a), p.ids(b), err_flag=p.err)
        p.host_fork(a, b)
    torch.cuda.synchronize()
    assert p.err.item() == 0 and not base[1::2].any()
    p.cache = p.cache.contiguous()
    p.same()


def test_page_refusals():
    p = Pool([40], 2)
    with pytest.raises(MlaError):
        p.fork([0], [1], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(MlaError):
        p.fork([0, 0, 0, 0], [1, 2, 1, 2])       # more pairs than rows
    with pytest.raises(TypeError):
        api.mla_kv_free(p.table.long(), p.lens, p.refs, p.ids([0]), block_size=16)
    with pytest.raises(MlaError):
        api.mla_kv_free(p.table, p.lens, p.refs, p.ids([0]), block_size=48)
    with pytest.raises(ValueError):
        api.mla_kv_fork(p.cache[:, :5], p.table, p.lens, p.refs, p.ids([0]), p.ids([1]))
    with pytest.raises(ValueError):
        api.mla_kv_copy_pages(p.cache, p.cache[:1], p.ids([0]), p.ids([1]))
    p.fork([], [])
    p.same()


def test_calls_in_a_row_see_each_others_writes():
    """Append, copy, append, fork and free back to back, each launched while the one
    before runs: the same bytes as with a wait after every call."""
    T, bs, layers = 40, 16, 1
    g = torch.Generator(device=DEV).manual_seed(5)
    kv = torch.randn(30, T, 576, generator=g, device=DEV).to(torch.bfloat16)
    cs = torch.randn(64, 64, generator=g, device=DEV)
    pos = torch.randint(0, 64, (T,), generator=g, device=DEV).int()
    ids = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    src, dst, p0, p1 = ids(0, 1, 2), ids(8, 9, 10), ids(0), ids(1)

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        pool = torch.zeros(layers, 14, bs, 324, dtype=torch.uint8, device=DEV)
        table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
        table[0, :3] = ids(8, 9, 10)
        lens, refs, err = ids(T, 0), torch.zeros(14, dtype=torch.int32, device=DEV), ids(0)
        refs[8:11] = 1
        refs[:3] = 1
        slots, seen = torch.arange(T, device=DEV).int(), []
        torch.cuda.synchronize()
        for k in range(30):
            api.mla_kv_append(kv[k][:, :512], kv[k][:, 512:], pool[0], slots, pos, cs, kv_scale=0.25, err_flag=err)
            sync()
            api.mla_kv_copy_pages(pool, pool, src, dst, err_flag=err)
            sync()
            api.mla_kv_fork(pool, table, lens, refs, p0, p1, err_flag=err)
            sync()
            seen.append((pool.clone(), table.clone(), refs.clone()))
            api.mla_kv_free(table, lens, refs, p1, block_size=bs, err_flag=err)
            sync()
        torch.cuda.synchronize()
        assert err.item() == 0
        return seen

    for a, b in zip(run(False), run(True)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
