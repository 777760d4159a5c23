"""Plain 64-bit forms of the cache operators for their tests: E2M1 rows and
pages, the append's rows, attention over given token values.  Written from the
formats and formulas; numpy only."""
import numpy as np

from oracle import mla_oracle as om

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = om.e4m3_to_f64(np.arange(256, dtype=np.uint8))


def nearest(x, grid):
    """Index of the grid value nearest to each x >= 0 (ties to the even index,
    past the end the last one).  grid ascending from 0."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def e4m3_bytes(x):
    """Nearest E4M3 bytes, saturating; NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    idx = nearest(np.minimum(np.abs(np.nan_to_num(x)), 448.0), E4M3[:127])
    out = idx.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), out)


def e2m1_rows(rows, kv_scale):
    """codes [..., 288], scales [..., 36] of rows [..., 576] (64 bits)."""
    rows = np.asarray(rows, np.float64)
    g = rows.reshape(*rows.shape[:-1], 36, 16)
    with np.errstate(invalid="ignore"):
        s = e4m3_bytes(np.abs(g).max(-1) / (6.0 * kv_scale))
    d = (E4M3[s] * kv_scale)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        m = nearest(np.where(d > 0, np.abs(g) / np.where(d > 0, d, 1.0), 0.0), MAGS)
    code = (m.astype(np.uint8) | (np.signbit(g).astype(np.uint8) << 3)).reshape(rows.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def e2m1_values(codes, scales, kv_scale):
    """Values [..., 576] of codes [..., 288] and scales [..., 36]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 576)
    v = MAGS[nib & 7] * np.where(nib >> 3, -1.0, 1.0)
    v = v.reshape(*codes.shape[:-1], 36, 16) * (E4M3[scales] * kv_scale)[..., None]
    return v.reshape(*codes.shape[:-1], 576)


def e2m1_pages(codes, scales):
    """[n, bs, 288], [n, bs, 36] -> pages [n, bs, 324]: all codes, then all scales."""
    n, bs = codes.shape[:2]
    return np.concatenate([codes.reshape(n, -1), scales.reshape(n, -1)], 1).reshape(n, bs, 324)


def split_pages(pages):
    n, bs = pages.shape[:2]
    flat = pages.reshape(n, -1)
    return flat[:, :bs * 288].reshape(n, bs, 288), flat[:, bs * 288:].reshape(n, bs, 36)


def rotate(v, cos, sin, interleaved):
    """Rotate [..., 64] pair by pair; cos, sin broadcast to [..., 32]."""
    v = np.asarray(v, np.float64)
    out = np.empty(v.shape)
    a, b = (v[..., 0::2], v[..., 1::2]) if interleaved else (v[..., :32], v[..., 32:])
    x, y = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        out[..., 0::2], out[..., 1::2] = x, y
    else:
        out[..., :32], out[..., 32:] = x, y
    return out


def append_rows(c_kv, k_pe, weight, eps, positions, sections, cos_sin, interleaved):
    """Rows [T, 576] in 64 bits, and each token's cos, sin [T, 32]."""
    c = np.asarray(c_kv, np.float64)
    lat = c if weight is None else c / np.sqrt((c * c).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight
    axis = np.repeat(np.arange(len(sections)), sections)
    table = np.asarray(cos_sin, np.float64)
    pair = np.arange(32)
    pos = positions[axis].T                                   # [T, 32]
    cos, sin = table[pos, pair], table[pos, 32 + pair]
    return np.concatenate([lat, rotate(k_pe, cos, sin, interleaved)], -1), cos, sin


def attention_parts(q_abs, q_pe, hist, cur, scale, shards, bs):
    """Partials of one sequence: q_abs [q, H, 512], hist [L, 576], cur [q, 576]
    or None (64 bits) -> o [q, P, H, 512], lse [q, P, H]."""
    n_q, H = q_abs.shape[:2]
    P = shards + (cur is not None)
    o, lse = np.zeros((n_q, P, H, 512)), np.full((n_q, P, H), -np.inf)
    for i in range(n_q):
        for p, (lo, hi) in enumerate(om.shard_bounds(len(hist), shards, bs)):
            o[i, p], lse[i, p] = om.segment_attention(q_abs[i], q_pe[i], hist[lo:hi], scale)
        if cur is not None:
            o[i, shards], lse[i, shards] = om.segment_attention(q_abs[i], q_pe[i], cur[:i + 1], scale)
    return o, lse
