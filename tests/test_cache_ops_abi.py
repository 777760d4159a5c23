"""Host-side argument checks of the cache operators (no GPU): bad calls are
refused before anything is launched.  And the tests' own 64-bit forms against
the formats."""
import ctypes

import numpy as np
import pytest

from mla_decode_attention_kv_gb300 import _ffi, build

import cache_util as cu

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    return _ffi.lib(build.build())


def _append(lib, **over):
    a = dict(c=FAKE, cs=576, k=FAKE, ks=576, w=FAKE, eps=1e-6, q=FAKE, qs=1024, qh=64, pos=FAKE, axes=1, sec=[32],
             table=FAKE, mp=100, inter=1, slots=FAKE, T=4, H=16, nb=10, bs=32, dt=0, fmt=2, scale=1.0, cache=FAKE,
             qo=FAKE, qos=1024, qoh=64, kv=None)
    a.update(over)
    sec = None if a["sec"] is None else (ctypes.c_int32 * len(a["sec"]))(*a["sec"])
    return lib.mla_kv_append(a["c"], a["cs"], a["k"], a["ks"], a["w"], a["eps"], a["q"], a["qs"], a["qh"], a["pos"],
                             a["axes"], sec, a["table"], a["mp"], a["inter"], a["slots"], a["T"], a["H"], a["nb"],
                             a["bs"], a["dt"], a["fmt"], a["scale"], a["cache"], a["qo"], a["qos"], a["qoh"], a["kv"],
                             None, None)


@pytest.mark.parametrize("over,status", [
    (dict(c=None), 1), (dict(cache=None), 1), (dict(qo=None), 1), (dict(q=None), 1), (dict(sec=None), 1),
    (dict(dt=2), 3), (dict(fmt=3), 3), (dict(fmt=-1), 3),
    (dict(T=0), 2), (dict(H=129), 2), (dict(H=0), 2), (dict(axes=4), 2), (dict(axes=0), 2), (dict(sec=[31]), 2),
    (dict(axes=2, sec=[40, -8]), 2), (dict(mp=0), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(scale=0.0), 2), (dict(scale=float("inf")), 2), (dict(scale=float("nan")), 2), (dict(cs=577), 2),
    (dict(ks=-8), 2), (dict(qh=60), 2), (dict(nb=1 << 28, bs=256), 2), (dict(T=1 << 30, H=128), 2), (dict(bs=48), 6), (dict(bs=0), 6),
    (dict(c=ODD), 4), (dict(w=ODD), 4), (dict(table=ODD), 4), (dict(kv=ODD), 4),
])
def test_append_host_checks(lib, over, status):
    assert _append(lib, **over) == status


def test_page_host_checks(lib):
    def fork(**o):
        a = dict(cache=FAKE, ls=1024, pb=512, L=2, t=FAKE, l=FAKE, r=FAKE, p=FAKE, c=FAKE, n=2, rows=8, nb=10, bs=16,
                 mb=4, ws=FAKE, wsb=1024)
        a.update(o)
        return lib.mla_kv_fork(a["cache"], a["ls"], a["pb"], a["L"], a["t"], a["l"], a["r"], a["p"], a["c"], a["n"],
                               a["rows"], a["nb"], a["bs"], a["mb"], a["ws"], a["wsb"], None, None)

    for o, st in ((dict(cache=None), 1), (dict(ws=None), 1), (dict(n=0), 2), (dict(n=9), 2), (dict(rows=65537), 2),
                  (dict(pb=8), 2), (dict(pb=520), 2), (dict(L=0), 2), (dict(L=65536), 2), (dict(ls=8), 2),
                  (dict(wsb=16), 2), (dict(mb=0), 2), (dict(bs=8), 6), (dict(r=ODD), 4), (dict(ws=ODD), 4),
                  (dict(pb=1 << 30, L=60000, n=8), 2)):
        assert fork(**o) == st, o
    assert lib.mla_kv_fork_workspace_size(0) == 0 and lib.mla_kv_fork_workspace_size(65537) == 0
    assert lib.mla_kv_fork_workspace_size(3) >= 40
    assert lib.mla_kv_free(FAKE, FAKE, None, FAKE, 1, 4, 4, 16, 4, None, None) == 1
    assert lib.mla_kv_free(FAKE, FAKE, FAKE, FAKE, 0, 4, 4, 16, 4, None, None) == 2
    assert lib.mla_kv_free(FAKE, FAKE, FAKE, FAKE, 1, 4, 4, 20, 4, None, None) == 6
    copy = lambda src=FAKE, pb=512, n=1, ids=FAKE, dl=0: lib.mla_kv_copy_pages(  # noqa: E731
        src, 0, 4, FAKE, dl, 4, pb, 1, ids, FAKE, n, None, None)
    assert copy(src=None) == 1 and copy(ids=None) == 1 and copy(pb=500) == 2 and copy(n=0) == 2
    assert copy(dl=4) == 2 and copy(src=ODD) == 4


def test_fp4_host_checks(lib):
    def part(kv_scale=0.01, **o):
        a = dict(q=FAKE, kv=FAKE, cur=None, B=2, q_len=1, H=128, nb=10, bs=32, mb=5, S=2, scale=0.07, idt=0, pdt=0,
                 ws=None, slices=1)
        a.update(o)
        return lib.mla_dcp_decode_partial_fp4(a["q"], FAKE, a["kv"], FAKE, FAKE, a["cur"], a["B"], a["q_len"], a["H"],
                                              a["nb"], a["bs"], a["mb"], a["S"], a["scale"], kv_scale, a["idt"],
                                              a["pdt"], FAKE, FAKE, None, a["ws"], 0, a["slices"], None)

    for o, st in ((dict(q=None), 1), (dict(idt=2), 3), (dict(pdt=3), 3), (dict(H=129), 2), (dict(q_len=65), 2),
                  (dict(S=65), 5), (dict(bs=48), 6), (dict(kv=ODD), 4), (dict(cur=ODD), 4), (dict(slices=3), 2),
                  (dict(ws=ctypes.c_void_p(0x10010)), 4), (dict(kv_scale=0.0), 2), (dict(kv_scale=-1.0), 2),
                  (dict(kv_scale=float("nan")), 2), (dict(kv_scale=float("inf")), 2),
                  # past the kernel's 32-bit counts: tokens with a round of shards, units, tiles
                  (dict(mb=(1 << 26) - 2), 2), (dict(B=1 << 20, q_len=64, S=64), 2), (dict(B=1 << 16, mb=1 << 20), 2)):
        assert part(**o) == st, o
    assert lib.mla_dcp_decode_partial_fp4_workspace_size(0, 1, 2, 0) == 0
    assert lib.mla_dcp_decode_partial_fp4_workspace_size(2, 1, 65, 1) == 0


def test_device_error_strings(lib):
    seen = {lib.mla_device_error_string(c) for c in range(9)}
    assert len(seen) == 9 and b"unknown device error" not in seen


def test_e2m1_helper_against_the_format():
    """Every magnitude and tie of a code, and a round trip of representable rows."""
    assert list(cu.nearest([0, .25, .2501, .75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5, 5.01, 6, 100], cu.MAGS)) == \
        [0, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 7]
    r = np.random.default_rng(0)
    mags = cu.MAGS[r.integers(0, 8, (5, 36, 16))]
    mags[..., 3] = 6.0
    rows = (mags * np.where(r.random(mags.shape) < .5, -1, 1) * 0.25 * 2.0 ** r.integers(-3, 4, (5, 36, 1))).reshape(5, 576)
    codes, scales = cu.e2m1_rows(rows, 0.25)
    assert np.array_equal(cu.e2m1_values(codes, scales, 0.25), rows)
    pages = cu.e2m1_pages(codes.reshape(5, 1, 288).repeat(16, 1), scales.reshape(5, 1, 36).repeat(16, 1))
    c, s = cu.split_pages(pages)
    assert pages.shape == (5, 16, 324) and np.array_equal(c[:, 3], codes) and np.array_equal(s[:, 15], scales)


def test_rotation_helper_keeps_lengths():
    r = np.random.default_rng(1)
    v, a = r.standard_normal((4, 64)), r.standard_normal((4, 32))
    for inter in (True, False):
        out = cu.rotate(v, np.cos(a), np.sin(a), inter)
        assert np.allclose((out ** 2).sum(-1), (v ** 2).sum(-1))
        assert np.allclose(cu.rotate(out, np.cos(a), -np.sin(a), inter), v)
