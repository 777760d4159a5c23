"""The partial call over an E2M1 cache with a block table wider than any history, as a
server that keeps one table has it: other work splits than the narrow table's, the same
answers.  Sizes, heads, pages and shards drawn."""
import random

import pytest
import torch

from test_gpu_fp4 import DEV, Fp4
from test_gpu_fp4_merge import check_rows

pytestmark = pytest.mark.gpu


def _widen(c, extra):
    B = c.gtable.shape[0]
    c.gtable = torch.cat([c.gtable, torch.full((B, extra), -1, dtype=torch.int32, device=DEV)], 1).contiguous()


@pytest.mark.parametrize("H", [1, 16, 17, 64, 65, 128])
@pytest.mark.parametrize("lens", [[0], [1], [64], [256], [65, 0, 1], [0, 0, 700], [512] * 8])
def test_short_histories_under_a_wide_table(H, lens):
    for cur in (False, True):
        c = Fp4(lens, H, shards=2, bs=16, cur=cur, seed=len(lens))
        narrow = c.run()
        _widen(c, 8192)
        o, lse = c.run()
        c.check(o, lse)
        check_rows(c, o)
        # (where no shard is cut either way the same units do the same sums)
        assert torch.equal(torch.isneginf(lse), torch.isneginf(narrow[1]))


@pytest.mark.parametrize("seed", range(40))
def test_drawn_sizes(seed):
    r = random.Random(seed)
    H = r.choice([r.randint(1, 128), 8, 16, 32, 64, 128])
    q_len = r.choice([1, 1, 1, 2, 3, 5])
    B = r.randint(1, 12)
    top = r.choice([3, 70, 400, 3000])
    lens = [r.choice([0, 1, r.randint(0, top), top]) for _ in range(B)]
    c = Fp4(lens, H, q_len=q_len, shards=r.choice([1, 2, 3, 7, 16, 64]), bs=r.choice([16, 32, 64, 128, 256]),
            cur=r.random() < .5, dtype=r.choice(["bf16", "fp16"]), part=r.choice(["bf16", "fp16", "fp32"]), seed=seed,
            gain=r.choice([0.3, 1.0, 3.0]), kv_scale=r.choice([2.0 ** -4, 0.011, 1.0]))
    if r.random() < .6:
        _widen(c, r.choice([1, 5, 300, 4000]))
    slices = r.choice([s for s in range(1, H + 1) if H % s == 0])
    o, lse = c.run()
    c.check(o, lse)
    check_rows(c, o)
    o2, l2 = c.run(head_slices=slices)
    P = o.shape[2]
    if slices > 1:
        assert torch.equal(o.reshape(B * q_len, P, slices, H // slices, 512).permute(2, 0, 1, 3, 4), o2)
        assert torch.equal(lse.reshape(B * q_len, P, slices, H // slices).permute(2, 0, 1, 3), l2)
    o3, l3 = c.run(workspace=None)
    c.check(o3, l3)
    check_rows(c, o3)
