"""The partial call over an E2M1 cache (mla_dcp_decode_partial_fp4) against
attention in 64 bits over the decoded pages.

Tolerances.  The products q k of 16-bit values are exact in fp32, a sum of 576
of them is off by at most 576 2^-24 sum|q k|, so a score by
D = scale 576 2^-24 max_t sum|q k| and the LSE by D and the rounding of a few
fp32 operations on it.  Softmax weights are rounded to 16 bits (half a step
h = eps / 2), then the output: o is off by (e^(2D) - 1 + h (1 + 2^-6)) max|c| +
h max|o|, and by the kernel's own fp32 sums, below h max|c| / 64 for these
lengths."""
import numpy as np
import pytest
import torch

from mla_decode_attention_kv_gb300 import api, inputs
from mla_decode_attention_kv_gb300._ffi import MlaError
from oracle import mla_oracle as om

import cache_util as cu
from gpu_util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TDT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


class Fp4:
    def __init__(self, lens, H, q_len=1, shards=2, bs=32, cur=False, dtype="bf16", part=None, seed=0, gain=1.0,
                 kv_scale=2.0 ** -4, stale=None):
        r = np.random.default_rng(seed)
        self.lens, self.H, self.q_len, self.S, self.bs, self.kv_scale = np.array(lens, np.int32), H, q_len, shards, bs, kv_scale
        self.dtype, self.part = dtype, TDT[part or dtype]
        B = len(lens)
        per = -(-self.lens // bs)
        blocks = max(1, int(per.sum()))
        rows = r.standard_normal((blocks, bs, 576)) * np.exp(0.4 * r.standard_normal(576))
        codes, scales = cu.e2m1_rows(rows, kv_scale)
        perm, at = r.permutation(blocks), 0
        self.table = np.full((B, max(1, int(per.max()))), -1, np.int32)
        self.hist = []
        for b in range(B):
            n, L = int(per[b]), int(self.lens[b])
            ids = perm[at:at + n]
            self.table[b, :n] = ids
            at += n
            vals = cu.e2m1_values(codes[ids].reshape(-1, 288), scales[ids].reshape(-1, 36), kv_scale)
            self.hist.append(vals[:L])
            if stale is not None and L % bs:
                codes[ids[-1], L % bs:] = stale
                scales[ids[-1], L % bs:] = stale
        dt = TDT[dtype]
        t = lambda *s: torch.from_numpy(r.standard_normal(s) * gain).to(dt).to(DEV)  # noqa: E731
        self.q_abs, self.q_pe = t(B, q_len, H, 512), t(B, q_len, H, 64)
        self.kv_cur = t(B, q_len, 576) / gain if cur else None
        self.pages = torch.from_numpy(cu.e2m1_pages(codes, scales)).to(DEV)
        self.gtable, self.glens = torch.from_numpy(self.table).to(DEV), torch.from_numpy(self.lens).to(DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        kw.setdefault("part_dtype", self.part)
        return api.mla_dcp_decode_partial(self.q_abs, self.q_pe, self.pages, self.gtable, self.glens, self.S,
                                          kv_cur=self.kv_cur, kv_scale=self.kv_scale, err_flag=self.err, **kw)

    def check(self, o, lse, batch=None):
        torch.cuda.synchronize()
        assert self.err.item() == 0
        scale = api.DEFAULT_SCALE
        qa, qp, go, gl = f64(self.q_abs), f64(self.q_pe), f64(o), f64(lse)
        half = float(torch.finfo(TDT[self.dtype]).eps) / 2
        oh = float(torch.finfo(self.part).eps) / 2
        for b in range(len(self.lens)) if batch is None else batch:
            cur = None if self.kv_cur is None else f64(self.kv_cur[b])
            ro, rl = cu.attention_parts(qa[b], qp[b], self.hist[b], cur, scale, self.S, self.bs)
            toks = self.hist[b] if cur is None else np.concatenate([self.hist[b], cur])
            q = np.abs(np.concatenate([qa[b], qp[b]], -1)).reshape(-1, 576)
            most = float((q @ np.abs(toks).T).max()) if len(toks) else 0.0
            D = scale * 576 * 2.0 ** -24 * most
            c = float(np.abs(toks[:, :512]).max()) if len(toks) else 0.0
            assert np.array_equal(np.isneginf(gl[b]), np.isneginf(rl))
            fin = np.isfinite(rl)
            if fin.any():
                lt = D + 2.0 ** -20 * (1 + np.abs(rl[fin]).max())
                assert np.abs(gl[b][fin] - rl[fin]).max() <= lt
            tol = (np.expm1(2 * D) + half * (1 + 2.0 ** -5)) * c + oh * np.abs(ro).max()
            assert np.isfinite(go[b]).all()
            assert np.abs(go[b] - ro).max() <= tol, (b, np.abs(go[b] - ro).max(), tol)


CASES = {
    "one_token": dict(lens=[1], H=1),
    "heads16_cur": dict(lens=[256], H=16, bs=64, cur=True),
    "odd_heads_fp16": dict(lens=[100, 3, 64], H=7, shards=3, dtype="fp16", bs=16),
    "heads12_q3": dict(lens=[130, 65], H=12, q_len=3, cur=True, bs=64),
    "heads24": dict(lens=[200, 511], H=24, bs=128),
    "heads40_fp16_q2": dict(lens=[333, 40], H=40, q_len=2, dtype="fp16", cur=True),
    "heads64": dict(lens=[700], H=64, shards=5, bs=256),
    "heads100_fp32part": dict(lens=[90, 1], H=100, part="fp32", bs=16),
    "heads128": dict(lens=[1000, 300], H=128, shards=3),
    "heads128_q2_cur": dict(lens=[150, 90], H=128, q_len=2, cur=True, bs=16),
    "current64": dict(lens=[70, 0], H=3, q_len=64, cur=True),
    "peaked": dict(lens=[600, 999], H=16, gain=8.0),
    "peaked_fp16": dict(lens=[600], H=33, gain=8.0, dtype="fp16"),
    "one_shard": dict(lens=[2000, 5], H=16, shards=1),
    "many_shards": dict(lens=[500, 2000], H=16, shards=64, bs=16),
    "scale": dict(lens=[300], H=16, kv_scale=0.0123),
    "large_scale": dict(lens=[300], H=16, kv_scale=3.0, dtype="fp16"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_fp4_partials_match_64_bits(name):
    c = Fp4(seed=len(name), **CASES[name])
    c.check(*c.run())


@pytest.mark.parametrize("lens", [[0, 0], [1, 0], [63, 64], [65, 127], [128, 129], [0, 1000], [31, 32, 33]])
@pytest.mark.parametrize("cur", [False, True])
def test_fp4_edge_lengths(lens, cur):
    c = Fp4(lens, 16, shards=4, cur=cur, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("H", [16, 128])
def test_fp4_stale_slots_may_hold_nan_scales(H):
    """Slots past a history's end: scale bytes of NaN, codes of any value."""
    for stale in (0x7F, 0xFF):
        c = Fp4([70, 129, 5, 64], H, bs=64, stale=stale, seed=4)
        c.check(*c.run())


def test_fp4_growing_scores():
    """Scores that rise along the history by more than the lazy rescale's threshold,
    tile after tile."""
    c = Fp4([900], 16, shards=1, seed=6)
    grow = torch.linspace(0.02, 3.0, 29, device=DEV)
    sc = c.pages.view(29, -1)[:, 32 * 288:]
    for j, page in enumerate(c.table[0]):
        s = sc[page].view(torch.float8_e4m3fn).float() * grow[j]
        sc[page] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    pages = c.pages.cpu().numpy()
    codes, scales = cu.split_pages(pages)
    c.hist[0] = cu.e2m1_values(codes[c.table[0]].reshape(-1, 288), scales[c.table[0]].reshape(-1, 36), c.kv_scale)[:900]
    c.q_abs.copy_((torch.from_numpy(c.hist[0][-1][:512]) / 4).to(torch.bfloat16).to(DEV).expand_as(c.q_abs))
    c.check(*c.run())


@pytest.mark.parametrize("H", [1, 5, 24, 32, 64, 100])
@pytest.mark.parametrize("rise", [3.0, 12.0])
def test_fp4_growing_scores_of_some_rows(H, rise):
    """Scores that rise tile after tile, in steps or by jumps, for every third row; the
    others' stay flat."""
    c = Fp4([1500], H, shards=1, seed=21, kv_scale=2.0 ** -4)
    n = len(c.table[0])
    grow = torch.linspace(0.02, rise, n, device=DEV)
    grow[n // 3: n // 2] = 0.02                       # a dip between
    sc = c.pages.view(c.pages.shape[0], -1)[:, 32 * 288:]
    for j, page in enumerate(c.table[0]):
        sc[page] = (sc[page].view(torch.float8_e4m3fn).float() * grow[j]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes, scales = cu.split_pages(c.pages.cpu().numpy())
    c.hist[0] = cu.e2m1_values(codes[c.table[0]].reshape(-1, 288), scales[c.table[0]].reshape(-1, 36), c.kv_scale)[:1500]
    along = torch.from_numpy(c.hist[0][-1] / np.abs(c.hist[0][-1]).max() * 3).to(torch.bfloat16).to(DEV)
    c.q_abs[:, :, ::3] = along[:512]
    c.q_pe[:, :, ::3] = along[512:]
    c.check(*c.run())


@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_fp4_split_and_whole_shards(H):
    """One long shard a sequence, cut between blocks with a workspace, whole without."""
    c = Fp4([9000, 4000], H, shards=1, bs=64, cur=True, seed=7)
    o1, l1 = c.run()
    c.check(o1, l1)
    o2, l2 = c.run(workspace=None)
    c.check(o2, l2)
    # the same call again gives the same bits
    o3, l3 = c.run()
    assert torch.equal(o1, o3) and torch.equal(l1, l3)


def test_fp4_many_short_units():
    r = np.random.default_rng(8)
    c = Fp4(list(r.integers(0, 60, 300)), 16, shards=16, bs=16, seed=8)
    o, lse = c.run()
    c.check(o, lse, batch=range(0, 300, 7))
    assert torch.isfinite(o.float()).all()


def test_fp4_head_slices_are_the_same_rows():
    c = Fp4([300, 77], 128, q_len=2, cur=True, seed=9)
    o1, l1 = c.run()
    o2, l2 = c.run(head_slices=4)
    B, q, P, H, D = o1.shape
    assert torch.equal(o1.reshape(B * q, P, 4, H // 4, D).permute(2, 0, 1, 3, 4), o2)
    assert torch.equal(l1.reshape(B * q, P, 4, H // 4).permute(2, 0, 1, 3), l2)


def test_fp4_device_errors():
    c = Fp4([100, 200], 16)
    c.gtable[1, 1] = 10 ** 6
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 1
    c = Fp4([100, 200], 16)
    c.glens[0] = 10 ** 6
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 3
    c = Fp4([100, 200], 16)
    c.glens[0] = -5
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 3
    c = Fp4([100, 200], 16, seed=11)
    c.check(*c.run())


def test_fp4_pages_past_4_gb():
    """Page offsets past 2^32 bytes: a sequence on the last pages of a large pool."""
    c = Fp4([700], 16, bs=256, seed=16)
    blocks = (1 << 32) // (256 * 324) + 60
    pool = torch.zeros(blocks, 256, 324, dtype=torch.uint8, device=DEV)
    n = c.pages.shape[0]
    pool[blocks - n:] = c.pages
    c.pages = pool
    c.gtable += torch.where(c.gtable >= 0, blocks - n, 0).to(torch.int32)
    c.check(*c.run())


def test_fp4_shared_and_repeated_pages():
    """Sequences that share pages (a fork), and a page that stands twice in a row."""
    c = Fp4([128, 128], 24, bs=32, seed=17)
    c.table[1] = c.table[0][[0, 1, 1, 3]]
    c.gtable = torch.from_numpy(c.table).to(DEV)
    h = c.hist[0]
    c.hist[1] = np.concatenate([h[:64], h[32:64], h[96:]])
    c.check(*c.run())


def test_fp4_two_streams_at_once():
    """Calls on two streams with their default workspaces (one each)."""
    cs = [Fp4([5000, 300], 16, shards=1, seed=18), Fp4([4000], 128, shards=2, seed=19)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(4):
        for k in range(2):
            outs[k] = cs[k].run(stream=streams[k])
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check(*o)


def test_fp4_graph_stream_and_two_workspaces():
    """Two captured calls that replay at once on two streams, each with a workspace
    of its own."""
    cs = [Fp4([3000, 500], 16, shards=1, seed=12), Fp4([2500, 700], 64, shards=1, seed=13)]
    graphs, outs = [], []
    for c in cs:
        o, lse = c.run()
        need = api._ffi.lib().mla_dcp_decode_partial_fp4_workspace_size(2, 1, 1, 0)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(o_part=o, lse_part=lse, workspace=ws)
        graphs.append(g)
        outs.append((o, lse, ws))
        o.zero_()
        lse.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (o, lse, _) in zip(cs, outs):
        c.check(o, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,at", [(4, 3), (16, 511), (40, 256), (128, 100), (16, 575)])
def test_fp4_current_rows_before_a_bad_token_stay_clean(value, H, at):
    """A value of CURRENT token 2 that is not finite: query tokens 0 and 1 do not see
    it, the others answer NaN (or, a score of -inf, as without it)."""
    c = Fp4([70, 5], H, q_len=4, cur=True, seed=20, shards=1)
    o1, l1 = c.run()
    c.kv_cur[1, 2, at] = value
    o2, l2 = c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    assert torch.equal(o1[0], o2[0]) and torch.equal(l1[0], l2[0])
    assert torch.equal(o1[1, :2], o2[1, :2]) and torch.equal(l1[1, :2], l2[1, :2])
    assert torch.equal(o1[1, 2:, 0], o2[1, 2:, 0])     # (the history's part has no such token)
    if at < 512:
        assert torch.isnan(o2[1, 2:, 1]).all() and torch.isnan(l2[1, 2:, 1]).all()


def test_fp4_graphs_with_default_workspaces():
    """Graphs captured on one stream with the default workspace replay at once on two."""
    cs = [Fp4([3000, 500], 16, shards=1, seed=12), Fp4([2500, 700], 64, shards=1, seed=13)]
    graphs, outs, side = [], [], torch.cuda.Stream()
    for c in cs:
        o, lse = c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.run(o_part=o, lse_part=lse)
        graphs.append(g)
        outs.append((o, lse))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (o, lse), s, g in zip(outs, streams, graphs):
            with torch.cuda.stream(s):
                o.zero_()
                lse.zero_()
                g.replay()
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cs, outs):
        c.check(o, lse)


def test_fp4_decode_step_and_refusals():
    c = Fp4([300, 20], 16, cur=True, seed=14)
    W = torch.randn(16, 512, 128, device=DEV).to(torch.bfloat16)
    out = api.decode_step(c.q_abs, c.q_pe, c.pages, c.gtable, c.glens, W, 2, kv_cur=c.kv_cur, kv_scale=c.kv_scale)
    o, lse = c.run()
    ro, _ = om.lse_combine(f64(o), f64(lse))
    ref = om.v_up(ro.reshape(2, 16, 512), f64(W))
    h = 2.0 ** -8
    assert np.abs(f64(out) - ref).max() <= h * np.abs(ref).max() + 2.0 ** -12 * np.abs(ro).max() * np.abs(f64(W)).sum(1).max()
    with pytest.raises(TypeError):
        api.mla_dcp_decode_partial(c.q_abs, c.q_pe, c.pages, c.gtable, c.glens, 2, kv_cur=c.kv_cur.half())
    with pytest.raises(MlaError):
        api.mla_dcp_decode_partial(c.q_abs, c.q_pe, c.pages, c.gtable, c.glens, 2, kv_scale=-1.0)
    with pytest.raises(MlaError):
        c.run(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)[16:])


def test_append_then_attend():
    """The operators together: tokens appended to an E2M1 cache over several calls,
    a fork of the sequence, then attention over both rows."""
    H, T, bs, S, ks = 16, 100, 32, 2, 2.0 ** -4
    g = torch.Generator(device=DEV).manual_seed(1)
    dt = torch.bfloat16
    pool = torch.zeros(12, bs, 324, dtype=torch.uint8, device=DEV)
    table = torch.full((2, 5), -1, dtype=torch.int32, device=DEV)
    table[0, :4] = torch.tensor([7, 2, 9, 4], device=DEV)
    refs = torch.zeros(12, dtype=torch.int32, device=DEV)
    refs[table[0, :4].long()] = 1
    lens = torch.tensor([T, 0], dtype=torch.int32, device=DEV)
    ang = torch.arange(T, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device=DEV) / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    kv_a = torch.randn(T, 576, generator=g, device=DEV).to(dt)
    q = torch.randn(T, H, 64, generator=g, device=DEV).to(dt)
    w = torch.ones(512, dtype=dt, device=DEV)
    rows = []
    for a, e in ((0, 50), (50, 99), (99, 100)):
        tok = torch.arange(a, e, device=DEV)
        slots = table[0][tok // bs] * bs + (tok % bs).int()
        q_rot, kv = api.mla_kv_append(kv_a[a:e, :512], kv_a[a:e, 512:], pool, slots, tok.int(), cs, norm_weight=w,
                                      q_pe=q[a:e], kv_out="new", kv_scale=ks)
        rows.append(kv)
    api.mla_kv_fork(pool, table, lens, refs, torch.tensor([0], dtype=torch.int32, device=DEV),
                    torch.tensor([1], dtype=torch.int32, device=DEV))
    hist = f64(torch.cat(rows))
    q_abs = torch.randn(2, 1, H, 512, generator=g, device=DEV).to(dt)
    q_abs[1] = q_abs[0]
    q_pe = q_rot[-1:].view(1, 1, H, 64).repeat(2, 1, 1, 1)
    o, lse = api.mla_dcp_decode_partial(q_abs, q_pe, pool, table, lens, S, kv_scale=ks)
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])
    assert table[1, 3].item() == 0 and refs[0].item() == 1 and refs[7].item() == 2
    ro, rl = cu.attention_parts(f64(q_abs[0]), f64(q_pe[0]), hist, None, api.DEFAULT_SCALE, S, bs)
    c = np.abs(hist).max()
    assert np.abs(f64(lse[0]) - rl).max() <= 1e-4
    assert np.abs(f64(o[0]) - ro).max() <= 2.0 ** -8 * (1 + 2.0 ** -5) * c + 2.0 ** -8 * np.abs(ro).max() + 2e-4 * c
