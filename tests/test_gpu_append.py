"""mla_kv_append against its 64-bit form: stored bytes equal, 16-bit values the
nearest ones."""
import numpy as np
import pytest
import torch

from mla_decode_attention_kv_gb300 import api
from mla_decode_attention_kv_gb300._ffi import MlaError

import cache_util as cu
from gpu_util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def _table(max_pos, seed=0):
    freq = 10000.0 ** (-np.arange(32) / 32)
    ang = np.arange(max_pos)[:, None] * freq
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(DEV)


class Case:
    def __init__(self, T, H, kind, dt=BF, axes=1, interleaved=True, bs=16, seed=0, kv_scale=2.0 ** -4,
                 max_pos=5000, pad=True, weight=True, strided=True):
        g = torch.Generator().manual_seed(seed)
        self.T, self.H, self.kind, self.dt, self.bs, self.kv_scale = T, H, kind, dt, bs, kv_scale
        self.interleaved, self.sections = interleaved, {1: [32], 2: [11, 21], 3: [6, 13, 13]}[axes]
        blocks = -(-T // bs) + 2
        slots = torch.randperm(blocks * bs, generator=g)[:T].to(torch.int32)
        if pad and T > 2:
            slots[T // 3] = -1
        kv_a = (torch.randn(T, 576 + 8 * strided, generator=g) * torch.exp(torch.randn(576 + 8 * strided, generator=g))).to(dt)
        q = torch.randn(T, H, 192 if strided else 64, generator=g).to(dt)
        self.kv_a, self.q = kv_a.to(DEV), q.to(DEV)
        self.c_kv, self.k_pe, self.q_pe = self.kv_a[:, :512], self.kv_a[:, 512:576], self.q[:, :, -64:]
        self.weight = (1 + 0.3 * torch.randn(512, generator=g)).to(dt).to(DEV) if weight else None
        self.positions = torch.randint(0, max_pos, (axes, T), generator=g, dtype=torch.int32).to(DEV)
        self.cos_sin = _table(max_pos)
        self.slots = slots.to(DEV)
        w, cdt = {"model": (576, dt), "e4m3": (576, torch.uint8), "e2m1": (324, torch.uint8)}[kind]
        self.cache = torch.full((blocks, bs, w), 3, dtype=cdt, device=DEV)   # a pattern to be left alone
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        args = dict(norm_weight=self.weight, eps=1e-5, q_pe=self.q_pe, kv_out="new", interleaved=self.interleaved,
                    sections=self.sections, err_flag=self.err,
                    kv_scale=None if self.kind == "model" else self.kv_scale)
        args.update(kw)
        return api.mla_kv_append(self.c_kv, self.k_pe, self.cache, self.slots, self.positions, self.cos_sin, **args)

    def rows(self):
        return cu.append_rows(f64(self.c_kv), f64(self.k_pe), None if self.weight is None else f64(self.weight), 1e-5,
                              self.positions.cpu().numpy(), self.sections, f64(self.cos_sin), self.interleaved)

    def check(self, q_out, kv_out):
        rows, cos, sin = self.rows()
        slots = self.slots.cpu().numpy()
        at = slots >= 0
        half = float(torch.finfo(self.dt).eps) / 2
        tiny = float(torch.finfo(self.dt).smallest_normal) * 2 ** -11   # half a subnormal step is below this x 2
        # queries: fp32 products and sum (three roundings of the larger terms), then the output's rounding
        if q_out is not None:
            ref = cu.rotate(f64(self.q_pe), cos[:, None], sin[:, None], self.interleaved)
            big = np.abs(f64(self.q_pe)).max(-1, keepdims=True)
            assert np.all(np.abs(f64(q_out) - ref) <= half * np.abs(ref) + 3 * 2.0 ** -24 * 2 * big + tiny * 2 ** 11)
        stored = np.zeros(self.cache.shape[0] * self.bs, bool)
        stored[slots[at]] = True
        if self.kind == "model":
            assert np.all(np.abs(f64(kv_out) - rows) <= half * np.abs(rows) * (1 + 2.0 ** -20) + tiny * 2 ** 11)
            flat = self.cache.view(-1, 576)
            assert torch.equal(flat[self.slots[self.slots >= 0].long()], kv_out[self.slots >= 0])
            assert (f64(flat)[~stored] == 3).all()
            return
        if self.kind == "e4m3":
            want = cu.e4m3_bytes(rows / self.kv_scale)
            assert np.array_equal(kv_out.view(torch.uint8).cpu().numpy(), want)
            flat = self.cache.cpu().numpy().reshape(-1, 576)
            assert np.array_equal(flat[slots[at]], want[at]) and (flat[~stored] == 3).all()
            return
        codes, scales = cu.e2m1_rows(rows, self.kv_scale)
        gc, gs = cu.split_pages(self.cache.cpu().numpy())
        gc, gs = gc.reshape(-1, 288), gs.reshape(-1, 36)
        assert np.array_equal(gs[slots[at]], scales[at]) and np.array_equal(gc[slots[at]], codes[at])
        assert (gc[~stored] == 3).all() and (gs[~stored] == 3).all()
        vals = cu.e2m1_values(codes, scales, self.kv_scale)
        assert np.all(np.abs(f64(kv_out) - vals) <= half * np.abs(vals) * (1 + 2.0 ** -20))
        if float(np.log2(self.kv_scale)).is_integer():
            assert np.array_equal(f64(kv_out), vals)


@pytest.mark.parametrize("kind", ["model", "e4m3", "e2m1"])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,axes,bs", [(1, 1, 1, 16), (7, 5, 2, 32), (130, 16, 3, 64), (33, 128, 1, 256)])
def test_append_matches_64_bits(kind, dt, interleaved, T, H, axes, bs):
    c = Case(T, H, kind, dt, axes, interleaved, bs, seed=T + H)
    q_out, kv_out = c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    c.check(q_out, kv_out)


def test_append_large_chunk_stores_nearest_codes():
    """Millions of values: a value rounded in fp32 before its border would show."""
    c = Case(6000, 2, "e2m1", axes=3, interleaved=False, bs=64, seed=9)
    q_out, kv_out = c.run()
    c.check(q_out, kv_out)
    assert c.err.item() == 0


@pytest.mark.parametrize("kind", ["model", "e2m1"])
def test_append_without_norm_queries_or_outputs(kind):
    c = Case(9, 3, kind, weight=False, strided=False)
    q_out, kv_out = c.run(q_pe=None, kv_out=None)
    assert q_out is None and kv_out is None
    _, kv_out = c.run()
    c.check(None, kv_out)


def test_append_queries_in_place():
    c = Case(20, 8, "model")
    before = c.q.clone()
    want, _ = c.run()
    got, _ = c.run(q_out=c.q_pe)
    assert got.data_ptr() == c.q_pe.data_ptr() and torch.equal(c.q_pe, want)
    assert torch.equal(c.q[:, :, :128], before[:, :, :128])


def test_append_scale_that_is_no_power_of_two():
    """kv_scale 0.0123: the quotients round in fp32, so a code may fall one off
    where the value is within 2^-22 of a border; at most one in 10^4 here."""
    c = Case(64, 1, "e2m1", kv_scale=0.0123)
    _, kv_out = c.run()
    rows, _, _ = c.rows()
    codes, scales = cu.e2m1_rows(rows, float(np.float32(0.0123)))
    vals = cu.e2m1_values(codes, scales, float(np.float32(0.0123)))
    off = np.abs(f64(kv_out) - vals) > 2.0 ** -8 * np.abs(vals) * 1.01
    assert off.mean() <= 1e-4


def test_append_zero_rows_ties_and_saturation():
    """Rows without a norm that hit the borders: zeros of both signs, exact ties,
    values past the E4M3 scale's range, and a NaN."""
    c = Case(6, 1, "e2m1", weight=False, pad=False, kv_scale=1.0, max_pos=1, strided=False)
    c.kv_a.zero_()
    c.kv_a[1] = -0.0
    # max 6 -> s = 1: ties between codes go to the even one
    c.kv_a[2, :512] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6.],
                                   device=DEV, dtype=BF).repeat(32)
    c.kv_a[3, :512] = 1e5                        # 1e5 / 6 is past 448: s saturates, codes 6
    c.kv_a[4, :512] = 2.0 ** -12                 # s rounds to 0: codes 0
    c.kv_a[5, 17] = float("nan")
    _, kv_out = c.run()
    assert c.err.item() == 0
    gc, gs = cu.split_pages(c.cache.cpu().numpy())
    slots = c.slots.cpu().numpy()
    codes, scales = cu.e2m1_rows(c.rows()[0], 1.0)     # (the key of -0 turns into +0, -0 pairs)
    gc, gs = gc.reshape(-1, 288)[slots], gs.reshape(-1, 36)[slots]
    assert np.array_equal(gs, scales)
    assert np.array_equal(gc[:5], codes[:5])
    assert np.array_equal(gc[5, 16:], codes[5, 16:])       # the NaN's block: its codes mean nothing
    v = kv_out[5].float()
    assert torch.isnan(v[16:32]).all() and torch.isfinite(v[:16]).all() and torch.isfinite(v[32:]).all()
    assert (kv_out[3, :512] == 6 * 448).all() and (kv_out[4] == 0).all()


@pytest.mark.parametrize("kind", ["model", "e4m3", "e2m1"])
def test_append_zero_rows_without_eps(kind):
    """0 / sqrt(0 + 0) counts as 0 (padding rows), and other rows are normalised as ever."""
    c = Case(5, 2, kind, pad=False)
    c.kv_a[1] = 0
    c.kv_a[3] = -0.0
    _, kv_out = c.run(eps=0.0)
    v = kv_out.view(torch.uint8) & 0x7F if kind == "e4m3" else kv_out
    assert (v[[1, 3]] == 0).all()
    r = f64(c.c_kv)[[0, 2, 4]]
    ref = r / np.sqrt((r * r).mean(-1, keepdims=True)) * f64(c.weight)
    if kind == "e4m3":
        assert np.array_equal(kv_out.view(torch.uint8).cpu().numpy()[[0, 2, 4], :512], cu.e4m3_bytes(ref / c.kv_scale))
    elif kind == "model":
        assert np.all(np.abs(f64(kv_out)[[0, 2, 4], :512] - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -20))


def test_append_one_token_of_any_stride():
    """The stride of a dimension of one element means nothing."""
    a, b = Case(1, 1, "model", seed=3), Case(1, 1, "model", seed=3)
    b.c_kv = a.c_kv.clone().reshape(512, 1).t()
    b.k_pe = a.k_pe.clone().reshape(64, 1).t()
    b.q_pe = a.q_pe.clone().reshape(64, 1, 1).permute(1, 2, 0)
    assert b.c_kv.stride(0) == 1 and b.q_pe.stride(1) == 1
    (q1, kv1), (q2, kv2) = a.run(), b.run()
    assert torch.equal(q1, q2) and torch.equal(kv1, kv2) and torch.equal(a.cache, b.cache)


def test_append_far_slots():
    """Slots past 2^31 bytes into the pool (32-bit byte offsets would wrap)."""
    blocks = (1 << 31) // (256 * 324) + 40
    c = Case(3, 1, "e2m1", bs=256, pad=False)
    c.cache = torch.zeros(blocks, 256, 324, dtype=torch.uint8, device=DEV)
    n = blocks * 256
    c.slots = torch.tensor([n - 1, n - 257, 5], dtype=torch.int32, device=DEV)
    _, kv_out = c.run()
    codes, scales = cu.e2m1_rows(c.rows()[0], c.kv_scale)
    for t, s in enumerate([n - 1, n - 257, 5]):
        page = c.cache[s // 256].cpu().numpy()[None]
        gc, gs = cu.split_pages(page)
        assert np.array_equal(gc[0, s % 256], codes[t]) and np.array_equal(gs[0, s % 256], scales[t])


@pytest.mark.parametrize("kind", ["model", "e4m3", "e2m1"])
def test_append_bad_slots_and_positions(kind):
    c = Case(40, 4, kind, pad=False)
    c.slots[3] = c.cache.shape[0] * c.bs
    c.slots[5] = -2
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 4
    q = Case(40, 4, kind)
    q.positions[0, 7] = q.cos_sin.shape[0]
    q.run()
    torch.cuda.synchronize()
    assert q.err.item() == 5


def test_append_graph_and_stream():
    """Captured on a stream of its own and replayed on new inputs."""
    c = Case(17, 4, "e2m1")
    s = torch.cuda.Stream()
    c.run()
    torch.cuda.synchronize()
    q_out = torch.empty(c.T, c.H, 64, dtype=c.dt, device=DEV)
    kv_out = torch.empty(c.T, 576, dtype=c.dt, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run(q_out=q_out, kv_out=kv_out)
    c.kv_a.normal_()
    c.q.normal_()
    c.cache.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    c.check(q_out, kv_out)


def test_append_refusals():
    c = Case(8, 2, "e2m1")
    with pytest.raises(TypeError):
        c.run(norm_weight=c.weight.float())
    with pytest.raises(ValueError):
        c.run(sections=[16, 16])
    with pytest.raises(MlaError):
        c.run(sections=[31])
    with pytest.raises(MlaError):
        c.run(kv_scale=0.0)
    with pytest.raises(MlaError):
        c.run(eps=-1.0)
    with pytest.raises(ValueError):
        c.run(kv_out=torch.empty(7, 576, dtype=BF, device=DEV))
    with pytest.raises(TypeError):
        Case(8, 2, "model").run(kv_scale=2.0)
    c.slots = c.slots.long()
    with pytest.raises(TypeError):
        c.run()
