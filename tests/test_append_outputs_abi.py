"""Host checks of mla_kv_append's outputs and sections (no GPU): what would make its
writes race or its axes wrap is refused before anything is launched."""
import ctypes

import pytest

from mla_decode_attention_kv_gb300 import _ffi, build

FAKE, OTHER = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x900000)
BAD_SHAPE, PAST_THE_CHECK = 2, 4       # (an odd cache pointer stops an accepted call: nothing is launched)


@pytest.fixture(scope="module")
def lib():
    return _ffi.lib(build.build())


def _append(lib, T=4, H=16, qs=1024, qh=64, qos=1024, qoh=64, qo=OTHER, sections=(32,)):
    sec = (ctypes.c_int32 * len(sections))(*sections)
    return lib.mla_kv_append(FAKE, 576, FAKE, 576, FAKE, 1e-6, FAKE, qs, qh, FAKE, len(sections), sec, FAKE, 100, 1,
                             FAKE, T, H, 10, 32, 0, 2, 1.0, ctypes.c_void_p(0x10008), qo, qos, qoh, None, None, None)


@pytest.mark.parametrize("over", [
    dict(qos=0), dict(qoh=0), dict(qos=0, qoh=0), dict(qos=56), dict(qoh=56), dict(qos=1016), dict(qos=64, qoh=64),
    dict(qos=64, qoh=248), dict(qos=1 << 62, qoh=1 << 58, T=2, H=128), dict(T=1, qoh=0), dict(H=1, qos=0),
    dict(T=1 << 20, qos=64, qoh=(1 << 26) - 8),
])
def test_overlapping_rows_of_q_out_are_refused(lib, over):
    assert _append(lib, **over) == BAD_SHAPE


@pytest.mark.parametrize("over", [
    dict(), dict(qos=2048), dict(qos=1024 + 8, qoh=64), dict(qos=64, qoh=256), dict(qos=72, qoh=280), dict(T=1, qos=0),
    dict(H=1, qoh=0), dict(T=1, H=1, qos=0, qoh=0), dict(T=1 << 20, qos=64, qoh=1 << 26),
    dict(qs=0, qh=0), dict(qs=64, qh=256),
])
def test_rows_apart_are_taken(lib, over):
    assert _append(lib, **over) == PAST_THE_CHECK


def test_in_place_with_other_strides_is_refused(lib):
    assert _append(lib, qo=FAKE) == PAST_THE_CHECK
    assert _append(lib, qo=FAKE, qos=2048) == BAD_SHAPE
    assert _append(lib, qo=FAKE, qos=64, qoh=256) == BAD_SHAPE
    assert _append(lib, qo=FAKE, T=1, qos=0) == PAST_THE_CHECK
    assert _append(lib, qo=FAKE, T=1, qos=0, qoh=128) == BAD_SHAPE
    assert _append(lib, qo=FAKE, H=1, qoh=0) == PAST_THE_CHECK


@pytest.mark.parametrize("sections", [
    (2 ** 31 - 1, 2 ** 31 - 1, 34), (33, -1), (2 ** 31 - 1, -(2 ** 31 - 1) + 32), (40, 40, -48), (0, 0, 0), (16, 15)])
def test_sections_that_do_not_sum_to_32(lib, sections):
    assert _append(lib, sections=sections) == BAD_SHAPE


@pytest.mark.parametrize("sections", [(32,), (0, 32), (32, 0, 0), (0, 0, 32), (1, 30, 1)])
def test_sections_that_sum_to_32(lib, sections):
    assert _append(lib, sections=sections) == PAST_THE_CHECK
