"""Calls over rows of one cache format refuse pools of another, before anything is
launched (no GPU: the format is checked first)."""
import pytest
import torch

from mla_decode_attention_kv_gb300 import api

BF, HF, U8 = torch.bfloat16, torch.float16, torch.uint8
E2M1 = torch.zeros(4, 16, 324, dtype=U8)
E4M3 = torch.zeros(4, 16, 576, dtype=U8)


def _args(dtype=BF):
    q_abs, q_pe = torch.zeros(1, 1, 2, 512, dtype=dtype), torch.zeros(1, 1, 2, 64, dtype=dtype)
    return q_abs, q_pe, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)


def _noalloc(cache, dtype=BF):
    q_abs, q_pe, table, lens = _args(dtype)
    api.mla_dcp_decode_partial_noalloc(q_abs, q_pe, cache, table, lens, 1, o_part=torch.zeros(1, 1, 1, 2, 512, dtype=dtype),
                                       lse_part=torch.zeros(1, 1, 1, 2))


def _gather(cache):
    _, _, table, lens = _args()
    api.mla_gather_kv(cache, table, lens, 32)


def _partial(cache, dtype=BF):
    q_abs, q_pe, table, lens = _args(dtype)
    api.mla_dcp_decode_partial(q_abs, q_pe, cache, table, lens, 1)


@pytest.mark.parametrize("call", [_noalloc, _gather])
@pytest.mark.parametrize("cache", [E2M1, E4M3, E4M3.view(torch.float8_e4m3fn), torch.zeros(4, 16, 576)],
                         ids=["e2m1", "e4m3 bytes", "e4m3", "fp32"])
def test_16_bit_calls_refuse_other_formats(call, cache):
    with pytest.raises(TypeError):
        call(cache)


@pytest.mark.parametrize("call", [_noalloc, _gather, _partial])
@pytest.mark.parametrize("shape", [(4, 16, 324), (4, 16, 575), (4, 16, 512), (64, 576)])
def test_16_bit_rows_are_576_wide(call, shape):
    with pytest.raises(ValueError):
        call(torch.zeros(shape, dtype=BF))


@pytest.mark.parametrize("call", [_noalloc, _partial])
def test_16_bit_cache_in_the_queries_type(call):
    with pytest.raises(TypeError):
        call(torch.zeros(4, 16, 576, dtype=HF), BF)
    with pytest.raises(TypeError):
        call(torch.zeros(4, 16, 576, dtype=BF), HF)


@pytest.mark.parametrize("width", [323, 325, 512, 577])
def test_byte_pools_of_no_format(width):
    with pytest.raises(ValueError):
        _partial(torch.zeros(4, 16, width, dtype=U8))


def test_gather_refuses_a_short_destination():
    _, _, table, lens = _args()
    with pytest.raises(ValueError):
        api.mla_gather_kv(torch.zeros(4, 16, 576, dtype=BF), table, lens, 32, dst=torch.zeros(1, 31, 576, dtype=BF))
    with pytest.raises(ValueError):
        api.mla_gather_kv(torch.zeros(4, 16, 576, dtype=BF), table, lens, 32, dst=torch.zeros(1, 32, 576, dtype=U8))
