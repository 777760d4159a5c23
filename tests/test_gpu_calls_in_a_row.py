"""Runs of cache operators back to back, each launched while the one before runs, against
the same runs with a wait after every call."""
import pytest
import torch

from mla_decode_attention_kv_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _ids(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("H,L", [(16, 100), (128, 300), (24, 1200)])
def test_attention_directly_behind_fork_and_free(H, L):
    """Fork, attend, free, fork from another row, attend: the attention starts while the
    grid before it still writes the block table and the lengths that it reads."""
    bs, rows = 16, 4
    g = torch.Generator(device=DEV).manual_seed(H)
    pages = -(-L // bs)
    lens0 = [L, L - 37, 0, 0]
    blocks = 2 * pages + 8
    pool = torch.zeros(blocks, bs, 324, dtype=torch.uint8, device=DEV)
    rnd = torch.randint(0, 256, pool.shape, generator=g, device=DEV, dtype=torch.uint8)
    flat = pool.view(blocks, -1)
    flat.copy_(rnd.view(blocks, -1))
    flat[:, bs * 288:] = (flat[:, bs * 288:] % 24) + 40          # block scales between 2^-2 and 2
    first = pool.clone()
    q_abs = torch.randn(rows, 1, H, 512, generator=g, device=DEV).to(BF)
    q_pe = torch.randn(rows, 1, H, 64, generator=g, device=DEV).to(BF)
    perm = torch.randperm(blocks, generator=g, device=DEV).int()

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        pool.copy_(first)
        table = torch.full((rows, pages + 2), -1, dtype=torch.int32, device=DEV)
        refs = torch.zeros(blocks, dtype=torch.int32, device=DEV)
        at = 0
        for r, n in enumerate(lens0):
            k = -(-n // bs)
            table[r, :k] = perm[at:at + k]
            refs[perm[at:at + k].long()] = 1
            at += k
        lens, err = _ids(*lens0), _ids(0)
        parents = [_ids(0, 1), _ids(1, 0), _ids(1, 1), _ids(0, 0)]
        kids, outs = _ids(2, 3), []
        ws = [torch.empty(64, dtype=torch.uint8, device=DEV) for _ in parents]
        torch.cuda.synchronize()
        for k in range(40):
            api.mla_kv_fork(pool, table, lens, refs, parents[k % 4], kids, workspace=ws[k % 4], err_flag=err)
            sync()
            outs.append(api.mla_dcp_decode_partial(q_abs, q_pe, pool, table, lens, 2, kv_scale=0.25, err_flag=err))
            sync()
            api.mla_kv_free(table, lens, refs, kids, block_size=bs, err_flag=err)
            sync()
            outs.append(api.mla_dcp_decode_partial(q_abs, q_pe, pool, table, lens, 2, kv_scale=0.25, err_flag=err))
            sync()
        torch.cuda.synchronize()
        assert err.item() == 0
        return outs

    a, b = run(False), run(True)
    assert all(torch.equal(x, y) for u, v in zip(a, b) for x, y in zip(u, v))
    lse = a[1][1]                                     # after the free: rows 2 and 3 are empty
    assert torch.isneginf(lse[2:]).all() and torch.isfinite(lse[:2]).all()


def test_copies_and_frees_by_ids_that_the_call_before_moved():
    """A copy whose ids were copied just before, and a free whose rows were: pools of one
    page of ids stand in for a scheduler on the device."""
    n, blocks = 16, 64
    lists = torch.stack([torch.randperm(32, device=DEV)[:n].int() for _ in range(8)]).view(8, 1, n)
    src = torch.randint(0, 256, (blocks, 16, 324), dtype=torch.uint8, device=DEV)
    one, dst_ids = _ids(0), torch.arange(n, dtype=torch.int32, device=DEV)
    sel = [_ids(k) for k in range(8)]

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        ids = torch.zeros(1, 1, n, dtype=torch.int32, device=DEV)
        dst = torch.zeros(n, 16, 324, dtype=torch.uint8, device=DEV)
        table = torch.arange(32 * 2, dtype=torch.int32, device=DEV).view(32, 2)
        lens = torch.full((32,), 20, dtype=torch.int32, device=DEV)
        refs, err, outs = torch.ones(64, dtype=torch.int32, device=DEV), _ids(0), []
        torch.cuda.synchronize()
        for k in range(24):
            api.mla_kv_copy_pages(lists, ids, sel[k % 8], one, err_flag=err)
            sync()
            api.mla_kv_copy_pages(src, dst, ids.view(-1), dst_ids, err_flag=err)
            sync()
            if k >= 20:
                api.mla_kv_free(table, lens, refs, ids.view(-1), block_size=16, err_flag=err)
                sync()
            outs.append((dst.clone(), table.clone(), lens.clone(), refs.clone()))
        torch.cuda.synchronize()
        assert err.item() == 0
        return outs

    assert all(torch.equal(x, y) for u, v in zip(run(False), run(True)) for x, y in zip(u, v))


@pytest.mark.parametrize("part", [BF, torch.float32])
@pytest.mark.parametrize("cache", ["16-bit", "e2m1"])
def test_combine_directly_behind_the_partials(part, cache):
    """Partials and the combine with the V-up (its two forms) into the same buffers, other
    queries every step: the combine starts while the partials are written."""
    B, H, L, bs = 6, 64, 700, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    n = -(-L // bs)
    if cache == "e2m1":
        pool = torch.randint(0, 256, (B * n, bs * 324), generator=g, device=DEV, dtype=torch.uint8)
        pool[:, bs * 288:] = pool[:, bs * 288:] % 24 + 40
        pool = pool.view(B * n, bs, 324)
    else:
        pool = torch.randn(B * n, bs, 576, generator=g, device=DEV).to(BF)
    table = torch.randperm(B * n, generator=g, device=DEV).int().view(B, n)
    lens, err = torch.full((B,), L, dtype=torch.int32, device=DEV), _ids(0)
    W = torch.randn(H, 512, 128, generator=g, device=DEV).to(BF)
    qs = [(torch.randn(B, 1, H, 512, generator=g, device=DEV).to(BF), torch.randn(B, 1, H, 64, generator=g, device=DEV).to(BF))
          for _ in range(5)]

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        o = torch.zeros(B, 1, 4, H, 512, dtype=part, device=DEV)
        lse, outs = torch.zeros(B, 1, 4, H, device=DEV), []
        torch.cuda.synchronize()
        for k in range(40):
            api.mla_dcp_decode_partial(*qs[k % 5], pool, table, lens, 4, o_part=o, lse_part=lse, err_flag=err)
            sync()
            outs.append(api.mla_lse_combine_vup(o, lse, W, err_flag=err))
            sync()
            outs.append(api.mla_vup(o[:, :, 0].contiguous().to(BF), W, err_flag=err))
            sync()
        torch.cuda.synchronize()
        assert err.item() == 0
        return outs

    assert all(torch.equal(x, y) for x, y in zip(run(False), run(True)))
