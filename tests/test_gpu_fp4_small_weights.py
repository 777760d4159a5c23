"""Many small softmax weights beside a large one: what a long history's tail adds up to."""
import math

import pytest
import torch

from mla_decode_attention_kv_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _pages(L, bs, top):
    """One sequence: latents 0 and a RoPE key of 6 on channel 0 for token `top`, latents 1
    and keys of 0 for all others (codes 0x2 = 1, 0x7 = 6; block scales 1)."""
    n = -(-L // bs)
    codes = torch.zeros(n * bs, 288, dtype=torch.uint8, device=DEV)
    codes[:, :256] = 0x22
    codes[top, :256] = 0
    codes[top, 256] = 0x07
    scales = torch.full((n * bs, 36), 0x38, dtype=torch.uint8, device=DEV)
    pool = torch.empty(n, bs * 324, dtype=torch.uint8, device=DEV)
    pool[:, :bs * 288] = codes.view(n, -1)
    pool[:, bs * 288:] = scales.view(n, -1)
    return pool.view(n, bs, 324)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("log2w", [-25.3, -24.6, -21.5, -16.2])
@pytest.mark.parametrize("top", [0, 40000])
def test_tail_of_a_long_history(dtype, H, log2w, top):
    """65536 tokens in one piece; all but one have the weight 2^log2w of the largest.  The
    weights are off by half a step, or, in fp16, by 2^-32 of the largest at most.

    The fp32 sums count here, with so many equal terms.  Row sums: a lane of the 64 adds
    L / 64 of them, each addition off by at most 2^-24 of the lane's sum, which is at most
    the row's: (L / 64) 2^-24 of the sum.  O: an MMA adds 16 tokens to what is there, off
    by at most a last bit (2^-23) of it, as the tensor cores may cut off instead of
    rounding: (L / 16) 2^-23 of O."""
    L, bs = 65536, 64
    pool = _pages(L, bs, top)
    table = torch.arange(L // bs, dtype=torch.int32, device=DEV).view(1, -1)
    lens, err = torch.tensor([L], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    q_abs = torch.zeros(1, 1, H, 512, dtype=dtype, device=DEV)
    q_pe = torch.zeros(1, 1, H, 64, dtype=dtype, device=DEV)
    q_pe[..., 0] = -log2w * math.log(2) / 6 / api.DEFAULT_SCALE
    w = math.exp(-float(q_pe[0, 0, 0, 0]) * 6 * api.DEFAULT_SCALE)
    o, lse = api.mla_dcp_decode_partial(q_abs, q_pe, pool, table, lens, 1, part_dtype=torch.float32, err_flag=err,
                                        workspace=None)
    assert err.item() == 0
    ref = (L - 1) * w / (1 + (L - 1) * w)
    h = torch.finfo(dtype).eps / 2
    sums = L / 64 * 2.0 ** -24
    tol = h * ref * (1 + 2.0 ** -6) + (L * 2.0 ** -32 if dtype == torch.float16 else 0) + \
        (2.0 ** -17 + sums + L / 16 * 2.0 ** -23) * ref
    assert (o.double() - ref).abs().max().item() <= tol
    assert (lse.double() - math.log(1 / w + L - 1)).abs().max().item() <= 2.0 ** -17 + sums
