"""Python binding of the C ABI (include/mla_dcp.h) for torch CUDA tensors.

Argument marshalling only: every call checks shapes, allocates outputs the
caller did not pass (torch owns device memory), and hands raw pointers to the
CUDA library on the current (or given) stream.  No arithmetic of the method
happens here and there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _ffi

D_LATENT, D_ROPE, D_QK, D_V = 512, 64, 576, 128
E2M1_ROW = 324      # bytes of one token in an E2M1 page: 288 of codes, 36 of block scales
DEFAULT_SCALE = 1.0 / math.sqrt(128 + D_ROPE)

_TORCH_DT = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
_DT_TORCH = {v: k for k, v in _TORCH_DT.items()}


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _code(dtype: torch.dtype) -> int:
    try:
        return _ffi.DTYPE[_TORCH_DT[dtype]]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


_WORKSPACES = {}


def partial_workspace(device, B: int, q_len: int, num_shards: int, has_current: bool,
                      stream=None):
    """The default workspace of mla_dcp_decode_partial on `device` for calls on
    `stream` (one per (device, stream), grown as needed), or None for sizes
    the library rejects.  Calls on one stream run one after another, so they
    can share it; calls on different streams get different workspaces.  Two
    calls that may overlap in time on the same stream handle (graphs replayed
    concurrently, say) must pass workspaces of their own."""
    device = torch.device(device)
    with torch.cuda.device(device):
        need = int(_ffi.lib().mla_dcp_decode_partial_workspace_size(
            B, q_len, num_shards, 1 if has_current else 0))
        s = stream if stream is not None else torch.cuda.current_stream()
    if need == 0:
        return None      # invalid sizes: the call itself reports them
    key = (device.index, s.cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


def is_fp8_cache(kv_cache) -> bool:
    """An E4M3 cache: uint8 bytes or torch.float8_e4m3fn."""
    return kv_cache.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))


def is_fp4_cache(kv_cache) -> bool:
    """An E2M1 cache: uint8 pages of 324 bytes a token (288 of codes, 36 of scales)."""
    return kv_cache.dtype == torch.uint8 and kv_cache.shape[-1] == E2M1_ROW


def mla_dcp_decode_partial(q_abs, q_pe, kv_cache, block_table, seq_lens, num_shards: int, *,
                           kv_cur=None, scale: float = DEFAULT_SCALE, part_dtype=None,
                           o_part=None, lse_part=None, err_flag=None, stream=None,
                           workspace="default", head_slices: int = 1, kv_scale=None):
    """Partial attention of every (sequence, query token, shard [, CURRENT]).

    q_abs [B, q, H, 512], q_pe [B, q, H, 64], kv_cache [num_blocks, bs, 576],
    block_table [B, max_blocks] int32, seq_lens [B] int32 (history lengths),
    kv_cur [B, q, 576] or None.  A kv_cache of E4M3 bytes (torch.uint8 or
    torch.float8_e4m3fn; kv_cur likewise) goes to mla_dcp_decode_partial_fp8
    with kv_scale (default 1.0); one of E2M1 pages (torch.uint8 [num_blocks,
    bs, 324]; kv_cur then in the dtype of q_abs) to mla_dcp_decode_partial_fp4.
    Returns o_part [B, q, P, H, 512] and
    lse_part [B, q, P, H] (float32), P = num_shards + (kv_cur is not None);
    with head_slices = N > 1 they are [N, B*q, P, H/N, 512] and
    [N, B*q, P, H/N] (mla_dcp_decode_partial_sliced: block n is what rank n
    receives in a head-scattered all-to-all).
    workspace: "default" (one kept per device and stream, see
    partial_workspace), a uint8 CUDA tensor of at least
    mla_dcp_decode_partial_workspace_size bytes, or None (pairs of CTAs then
    take whole shards)."""
    if is_fp4_cache(kv_cache):
        return _partial_fp4(q_abs, q_pe, kv_cache, block_table, seq_lens, num_shards, kv_cur, scale,
                            part_dtype, o_part, lse_part, err_flag, stream, workspace, head_slices,
                            1.0 if kv_scale is None else kv_scale)
    B, q_len, H, _ = q_abs.shape
    num_blocks, bs, _ = kv_cache.shape
    P = num_shards + (1 if kv_cur is not None else 0)
    part_dtype = part_dtype or q_abs.dtype
    for t, n in ((q_abs, "q_abs"), (q_pe, "q_pe"), (kv_cache, "kv_cache"),
                 (block_table, "block_table"), (seq_lens, "seq_lens")):
        _need(t, n)
    if head_slices == 1:
        o_shape, l_shape = (B, q_len, P, H, D_LATENT), (B, q_len, P, H)
    else:
        hs = H // head_slices
        o_shape = (head_slices, B * q_len, P, hs, D_LATENT)
        l_shape = (head_slices, B * q_len, P, hs)
    if o_part is None:
        o_part = torch.empty(o_shape, dtype=part_dtype, device=q_abs.device)
    if lse_part is None:
        lse_part = torch.empty(l_shape, dtype=torch.float32, device=q_abs.device)
    if isinstance(workspace, str):
        if workspace != "default":
            raise ValueError("workspace must be 'default', a tensor or None")
        workspace = partial_workspace(q_abs.device, B, q_len, num_shards, kv_cur is not None,
                                      stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if is_fp8_cache(kv_cache):
        if kv_cur is not None and not is_fp8_cache(kv_cur):
            raise TypeError("kv_cur must be E4M3 bytes like kv_cache")
        st = _ffi.lib().mla_dcp_decode_partial_fp8(
            _p(q_abs), _p(q_pe), _p(kv_cache), _p(block_table), _p(seq_lens), _p(kv_cur),
            B, q_len, H, num_blocks, bs, block_table.shape[1], num_shards, float(scale),
            float(1.0 if kv_scale is None else kv_scale), _code(q_abs.dtype),
            _code(o_part.dtype), _p(o_part), _p(lse_part), _p(err_flag), _p(workspace), ws_bytes,
            int(head_slices), _s(stream))
        _ffi.check("mla_dcp_decode_partial_fp8", st)
        return o_part, lse_part
    if kv_scale is not None:
        raise TypeError("kv_scale applies to an E4M3 cache only")
    st = _ffi.lib().mla_dcp_decode_partial_sliced(
        _p(q_abs), _p(q_pe), _p(kv_cache), _p(block_table), _p(seq_lens), _p(kv_cur),
        B, q_len, H, num_blocks, bs, block_table.shape[1], num_shards, float(scale),
        _code(q_abs.dtype), _code(o_part.dtype), _p(o_part), _p(lse_part), _p(err_flag),
        _p(workspace), ws_bytes, int(head_slices), _s(stream))
    _ffi.check("mla_dcp_decode_partial_sliced", st)
    return o_part, lse_part


def mla_dcp_combine_exchanged(o_recv, lse_recv, *, hist_parts: int, local_src: int = -1,
                              out_dtype=None, o_latent=None, lse_out=None, stream=None):
    """Combine on one GPU after the head-scattered exchange: o_recv
    [N, T, P, Hs, 512] and lse_recv [N, T, P, Hs] as delivered by the
    all-to-all; parts p < hist_parts of every source plus (if local_src >= 0)
    part hist_parts of source local_src.  Returns o_latent [T, Hs, 512] and
    lse [T, Hs]."""
    N, T, P, Hs, _ = o_recv.shape
    _need(o_recv, "o_recv")
    _need(lse_recv, "lse_recv")
    out_dtype = out_dtype or o_recv.dtype
    if o_latent is None:
        o_latent = torch.empty((T, Hs, D_LATENT), dtype=out_dtype, device=o_recv.device)
    if lse_out is None:
        lse_out = torch.empty((T, Hs), dtype=torch.float32, device=o_recv.device)
    st = _ffi.lib().mla_dcp_combine_exchanged(
        _p(o_recv), _p(lse_recv), N, P, int(hist_parts), int(local_src), T, Hs,
        _code(o_recv.dtype), _code(o_latent.dtype), _p(o_latent), _p(lse_out), _s(stream))
    _ffi.check("mla_dcp_combine_exchanged", st)
    return o_latent, lse_out


def mla_dcp_decode_partial_noalloc(q_abs, q_pe, kv_cache, block_table, seq_lens,
                                   num_shards: int, *, o_part, lse_part, kv_cur=None,
                                   scale: float = DEFAULT_SCALE, err_flag=None, stream=None):
    """mla_dcp_decode_partial with the library's fixed scratch array instead of
    a workspace: allocates nothing (o_part / lse_part are required), for
    callers that cannot lend the library device memory.  Calls that may
    overlap in time share that array and must be serialised."""
    B, q_len, H, _ = q_abs.shape
    num_blocks, bs, _ = kv_cache.shape
    for t, n in ((q_abs, "q_abs"), (q_pe, "q_pe"), (kv_cache, "kv_cache"),
                 (block_table, "block_table"), (seq_lens, "seq_lens"), (o_part, "o_part"),
                 (lse_part, "lse_part")):
        _need(t, n)
    st = _ffi.lib().mla_dcp_decode_partial_noalloc(
        _p(q_abs), _p(q_pe), _p(kv_cache), _p(block_table), _p(seq_lens), _p(kv_cur),
        B, q_len, H, num_blocks, bs, block_table.shape[1], num_shards, float(scale),
        _code(q_abs.dtype), _code(o_part.dtype), _p(o_part), _p(lse_part), _p(err_flag),
        _s(stream))
    _ffi.check("mla_dcp_decode_partial_noalloc", st)
    return o_part, lse_part


def _rows(o_part, lse_part):
    """View [..., P, H, 512] partials as T rows."""
    P, H = o_part.shape[-3], o_part.shape[-2]
    T = o_part.numel() // (P * H * D_LATENT)
    return T, P, H


def mla_lse_combine(o_part, lse_part, *, o_local=None, lse_local=None, out_dtype=None,
                    o_latent=None, lse_out=None, stream=None):
    """LSE-weighted merge of partials [..., P, H, 512] (+ optional local
    [..., H, 512]) -> o_latent [T, H, 512], lse [T, H]."""
    T, P, H = _rows(o_part, lse_part)
    _need(o_part, "o_part")
    _need(lse_part, "lse_part")
    out_dtype = out_dtype or o_part.dtype
    if o_latent is None:
        o_latent = torch.empty((T, H, D_LATENT), dtype=out_dtype, device=o_part.device)
    if lse_out is None:
        lse_out = torch.empty((T, H), dtype=torch.float32, device=o_part.device)
    st = _ffi.lib().mla_lse_combine(
        _p(o_part), _p(lse_part), P, _p(o_local), _p(lse_local), T, H, _code(o_part.dtype),
        _code(o_latent.dtype), _p(o_latent), _p(lse_out), _s(stream))
    _ffi.check("mla_lse_combine", st)
    return o_latent, lse_out


def mla_vup(o_latent, W_UV, *, out=None, err_flag=None, stream=None):
    """out [T, H*128] = per-head o_latent[:, h, :] @ W_UV[h]."""
    H = W_UV.shape[0]
    T = o_latent.numel() // (H * D_LATENT)
    _need(o_latent, "o_latent")
    _need(W_UV, "W_UV")
    if out is None:
        out = torch.empty((T, H * D_V), dtype=W_UV.dtype, device=W_UV.device)
    st = _ffi.lib().mla_vup(_p(o_latent), _p(W_UV), T, H, _code(W_UV.dtype), _p(out),
                            _p(err_flag), _s(stream))
    _ffi.check("mla_vup", st)
    return out


def mla_lse_combine_vup(o_part, lse_part, W_UV, *, o_local=None, lse_local=None, out=None,
                        o_latent=None, lse_out=None, err_flag=None, stream=None):
    """Combine + V-up in one launch -> out [T, H*128] (and optionally the
    combined latent / LSE if o_latent / lse_out are given)."""
    T, P, H = _rows(o_part, lse_part)
    _need(o_part, "o_part")
    _need(W_UV, "W_UV")
    if out is None:
        out = torch.empty((T, H * D_V), dtype=W_UV.dtype, device=W_UV.device)
    st = _ffi.lib().mla_lse_combine_vup(
        _p(o_part), _p(lse_part), P, _p(o_local), _p(lse_local), _p(W_UV), T, H,
        _code(o_part.dtype), _code(W_UV.dtype), _p(out), _p(o_latent), _p(lse_out),
        _p(err_flag), _s(stream))
    _ffi.check("mla_lse_combine_vup", st)
    return out


def mla_gather_kv(kv_cache, block_table, seq_lens, max_len: int, *, dst=None, err_flag=None,
                  stream=None):
    """dst [B, max_len, 576]: each sequence's paged history, bit-exact."""
    B = block_table.shape[0]
    num_blocks, bs, _ = kv_cache.shape
    if dst is None:
        dst = torch.empty((B, max_len, D_QK), dtype=kv_cache.dtype, device=kv_cache.device)
    st = _ffi.lib().mla_gather_kv(_p(kv_cache), _p(block_table), _p(seq_lens), B, num_blocks, bs,
                                  block_table.shape[1], max_len, _p(dst), _p(err_flag),
                                  _s(stream))
    _ffi.check("mla_gather_kv", st)
    return dst


def decode_step(q_abs, q_pe, kv_cache, block_table, seq_lens, W_UV, num_shards: int, *,
                kv_cur=None, scale: float = DEFAULT_SCALE, part_dtype=None, o_part=None,
                lse_part=None, out=None, err_flag=None, stream=None, workspace="default",
                kv_scale=None):
    """One decode step of the attention layer: partials, then the fused
    combine + V-up.  Returns out [B*q, H*128]."""
    o_part, lse_part = mla_dcp_decode_partial(
        q_abs, q_pe, kv_cache, block_table, seq_lens, num_shards, kv_cur=kv_cur, scale=scale,
        part_dtype=part_dtype, o_part=o_part, lse_part=lse_part, err_flag=err_flag,
        stream=stream, workspace=workspace, kv_scale=kv_scale)
    return mla_lse_combine_vup(o_part, lse_part, W_UV, out=out, err_flag=err_flag, stream=stream)


# ---------------------------------------------------------------- cache operators
# Their calls can be as short as a launch, so their host side is kept short: raw
# pointers and stream handles, device ordinals instead of device objects, and
# the words of an error only once there is one.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _call(name: str, i: int, stream, *args):
    """Library call `name` on device i, on `stream` (default: the device's current one)."""
    fn = getattr(_ffi.lib(), name)
    s = _raw_stream(i) if stream is None else stream.cuda_stream
    if _current_device() == i:
        st = fn(*args, s)
    else:
        with torch.cuda.device(i):
            st = fn(*args, s)
    if st != 0:
        raise _ffi.MlaError(name, st)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _device(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _on(t: torch.Tensor, i: int, name: str, dtype=None):
    """A tensor on device i (the call's stream and launches are on that device)."""
    if t.get_device() != i:
        raise ValueError(f"{name} must be a CUDA tensor on device {i}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _dense(t: torch.Tensor, i: int, name: str, dtype, *shape):
    """A contiguous tensor of one shape and type on device i."""
    if t.get_device() != i or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _on(t, i, name, dtype)
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape}, not {tuple(t.shape)}")


def _err(t: Optional[torch.Tensor], i: int):
    if t is not None:
        _on(t, i, "err_flag", torch.int32)
        if t.numel() < 1:
            raise ValueError("err_flag must hold one int32")


def _partial_fp4(q_abs, q_pe, kv_cache, block_table, seq_lens, num_shards, kv_cur, scale,
                 part_dtype, o_part, lse_part, err_flag, stream, workspace, head_slices, kv_scale):
    """mla_dcp_decode_partial over E2M1 pages."""
    B, q_len, H, _ = q_abs.shape
    i, dt = _device(q_abs, "q_abs"), q_abs.dtype
    _dense(q_abs, i, "q_abs", dt, B, q_len, H, D_LATENT)
    _dense(q_pe, i, "q_pe", dt, B, q_len, H, D_ROPE)
    num_blocks, bs, _ = kv_cache.shape
    _dense(kv_cache, i, "kv_cache", torch.uint8, num_blocks, bs, E2M1_ROW)
    max_blocks = block_table.shape[-1]
    _dense(block_table, i, "block_table", torch.int32, B, max_blocks)
    _dense(seq_lens, i, "seq_lens", torch.int32, B)
    if kv_cur is not None:
        _dense(kv_cur, i, "kv_cur", dt, B, q_len, D_QK)
    _err(err_flag, i)
    P = num_shards + (kv_cur is not None)
    o_rows = ((B, q_len, P, H) if head_slices == 1
              else (head_slices, B * q_len, P, H // max(1, head_slices)))
    if o_part is None:
        o_part = torch.empty(o_rows + (D_LATENT,), dtype=part_dtype or dt, device=q_abs.device)
    else:
        _dense(o_part, i, "o_part", part_dtype or o_part.dtype, *o_rows, D_LATENT)
    if lse_part is None:
        lse_part = torch.empty(o_rows, dtype=torch.float32, device=q_abs.device)
    else:
        _dense(lse_part, i, "lse_part", torch.float32, *o_rows)
    if isinstance(workspace, str):
        if workspace != "default":
            raise ValueError("workspace must be 'default', a tensor or None")
        workspace = _fp4_workspace(i, B, q_len, num_shards, kv_cur is not None, stream)
    elif workspace is not None:
        _on(workspace, i, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _call("mla_dcp_decode_partial_fp4", i, stream, q_abs.data_ptr(), q_pe.data_ptr(),
          kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), _ptr(kv_cur), B, q_len, H,
          num_blocks, bs, max_blocks, num_shards, scale, kv_scale, _code(dt), _code(o_part.dtype),
          o_part.data_ptr(), lse_part.data_ptr(), _ptr(err_flag), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), head_slices)
    return o_part, lse_part


_FP4_WORKSPACES = {}


def _fp4_workspace(i: int, B: int, q_len: int, num_shards: int, has_current: bool, stream):
    """The default workspace of mla_dcp_decode_partial_fp4 (see partial_workspace): one per
    (device, stream); its size depends on the device alone."""
    key = (i, _raw_stream(i) if stream is None else stream.cuda_stream)
    ws = _FP4_WORKSPACES.get(key)
    if ws is None:
        with torch.cuda.device(i):
            need = int(_ffi.lib().mla_dcp_decode_partial_fp4_workspace_size(
                B, q_len, num_shards, 1 if has_current else 0))
            if need == 0:
                return None      # invalid sizes: the call itself reports them
            ws = torch.empty(need, dtype=torch.uint8, device=f"cuda:{i}")
        _FP4_WORKSPACES[key] = ws
    return ws


def _kv_format(kv_cache: torch.Tensor, dtype: torch.dtype) -> str:
    """Storage of a paged cache [num_blocks, bs, W] for a model dtype."""
    if kv_cache.dim() != 3 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [num_blocks, block_size, W] tensor")
    if is_fp4_cache(kv_cache):
        return "e2m1"
    if kv_cache.shape[2] == D_QK:
        if kv_cache.dtype == dtype:
            return "model"
        if is_fp8_cache(kv_cache):
            return "e4m3"
    raise TypeError(f"no cache format has rows of {kv_cache.shape[2]} x {kv_cache.dtype} for {dtype}")


_SECTIONS = {}     # position sections as C arrays


def mla_kv_append(c_kv, k_pe, kv_cache, slots, positions, cos_sin, *, norm_weight=None,
                  eps: float = 1e-6, q_pe=None, q_out=None, kv_out=None, kv_scale=None,
                  interleaved: bool = True, sections=(D_ROPE // 2,), err_flag=None, stream=None):
    """Norm, rotate and store new tokens, and rotate their queries, in one launch.

    c_kv [T, 512] and k_pe [T, 64] (rows may be strided: views of one
    projection), kv_cache [num_blocks, bs, 576] in their dtype or as E4M3
    bytes, or [num_blocks, bs, 324] uint8 E2M1 pages (kv_scale, default 1.0,
    for the last two), slots [T] int32 (-1: store nowhere), positions [T] or
    [axes, T] int32, cos_sin [max_pos, 64] float32 (32 cosines, 32 sines),
    norm_weight [512] or None (no norm), q_pe [T, H, 64] (strided) or None.
    sections: pairs of each axis, sum 32 (default: all 32 on one axis).
    q_out: rotated queries, a new [T, H, 64] tensor if None, may be q_pe.
    kv_out: None, "new" or a [T, 576] tensor: the rows as the partial call's
    kv_cur (16-bit; E4M3 bytes for an E4M3 cache; over an E2M1 cache the values
    that were stored).  Returns (q_out, kv_out)."""
    i, dt = _device(c_kv, "c_kv"), c_kv.dtype
    T, w = c_kv.shape
    (cs, c1), (ks, k1) = c_kv.stride(), k_pe.stride()
    if w != D_LATENT or k_pe.shape != (T, D_ROPE) or c1 != 1 or k1 != 1:
        raise ValueError("c_kv must be [T, 512] and k_pe [T, 64] with unit stride along their rows")
    _on(k_pe, i, "k_pe", dt)
    _on(kv_cache, i, "kv_cache")
    fmt = _kv_format(kv_cache, dt)
    if fmt == "model" and kv_scale is not None:
        raise TypeError("kv_scale applies to an E4M3 or E2M1 cache only")
    _dense(slots, i, "slots", torch.int32, T)
    sections = tuple(sections)
    axes = len(sections)
    if positions.dim() == 1:
        _dense(positions, i, "positions", torch.int32, T)
        if axes != 1:
            raise ValueError(f"{axes} sections for one position axis")
    else:
        _dense(positions, i, "positions", torch.int32, axes, T)
    sec = _SECTIONS.get(sections)
    if sec is None:
        sec = _SECTIONS[sections] = (ctypes.c_int32 * axes)(*sections)
    max_pos = cos_sin.shape[0]
    _dense(cos_sin, i, "cos_sin", torch.float32, max_pos, D_ROPE)
    if norm_weight is not None:
        _dense(norm_weight, i, "norm_weight", dt, D_LATENT)
    _err(err_flag, i)
    H = qs = qh = os = oh = 0
    if q_pe is not None:
        H = q_pe.shape[1]
        qs, qh, q1 = q_pe.stride()
        _on(q_pe, i, "q_pe", dt)
        if q_pe.shape != (T, H, D_ROPE) or q1 != 1:
            raise ValueError("q_pe must be [T, H, 64] with unit stride along its heads")
        if q_out is None:
            q_out = torch.empty((T, H, D_ROPE), dtype=dt, device=c_kv.device)
            os, oh = H * D_ROPE, D_ROPE
        else:
            os, oh, q1 = q_out.stride()
            _on(q_out, i, "q_out", dt)
            if q_out.shape != (T, H, D_ROPE) or q1 != 1:
                raise ValueError("q_out must be [T, H, 64] with unit stride along its heads")
    elif q_out is not None:
        raise ValueError("q_out without q_pe")
    kv_dt = kv_cache.dtype if fmt == "e4m3" else dt
    if isinstance(kv_out, str):
        if kv_out != "new":
            raise ValueError("kv_out must be None, 'new' or a tensor")
        kv_out = torch.empty((T, D_QK), dtype=kv_dt, device=c_kv.device)
    elif kv_out is not None:
        _on(kv_out, i, "kv_out", kv_dt)
        if kv_out.numel() != T * D_QK or not kv_out.is_contiguous():
            raise ValueError("kv_out must be a contiguous [T, 576] tensor")
    if T > 0:
        _call("mla_kv_append", i, stream, c_kv.data_ptr(), cs, k_pe.data_ptr(), ks,
              _ptr(norm_weight), eps, _ptr(q_pe), qs, qh, positions.data_ptr(), axes,
              sec, cos_sin.data_ptr(), max_pos, 1 if interleaved else 0, slots.data_ptr(), T, H,
              kv_cache.shape[0], kv_cache.shape[1], _code(dt), _ffi.KV_FORMAT[fmt],
              1.0 if kv_scale is None else kv_scale, kv_cache.data_ptr(), _ptr(q_out), os, oh,
              _ptr(kv_out), _ptr(err_flag))
    return q_out, kv_out


def _pools(kv_cache: torch.Tensor, name: str):
    """(layers, layer stride in bytes, pages, bytes of a page, block size) of a pool
    [num_blocks, bs, W] or the layers' pools [layers, num_blocks, bs, W]."""
    shape = kv_cache.shape
    if len(shape) not in (3, 4):
        raise ValueError(f"{name} must be a tensor [(layers,) num_blocks, block_size, W]")
    size = kv_cache.element_size()
    n, bs, w = shape[-3:]
    if kv_cache.stride()[-3:] != (bs * w, w, 1):
        raise ValueError(f"the pages of {name} must be contiguous")
    layers = 1 if len(shape) == 3 else shape[0]
    stride = 0 if layers == 1 else kv_cache.stride(0) * size
    if layers > 1 and stride < n * bs * w * size:
        raise ValueError(f"the layers of {name} overlap")
    return layers, stride, n, bs * w * size, bs


def mla_kv_copy_pages(src, dst, src_ids, dst_ids, *, err_flag=None, stream=None):
    """Pages src_ids [n] of the pool(s) `src` to pages dst_ids [n] of `dst`, in every layer.
    Pools are [num_blocks, bs, W] or [layers, num_blocks, bs, W] of one format.  dst_ids are
    distinct, and within one pool no page is both source and destination.  Returns dst."""
    i = _device(src, "src")
    sl, ss, sn, sp, _ = _pools(src, "src")
    dl, ds, dn, dp, _ = _pools(dst, "dst")
    if sl != dl or sp != dp or src.dtype != dst.dtype:
        raise ValueError("src and dst must hold pages of one size and type in as many layers")
    n = src_ids.numel()
    _on(dst, i, "dst")
    _dense(src_ids, i, "src_ids", torch.int32, n)
    _dense(dst_ids, i, "dst_ids", torch.int32, n)
    _err(err_flag, i)
    if n > 0:
        _call("mla_kv_copy_pages", i, stream, src.data_ptr(), ss, sn, dst.data_ptr(), ds, dn, sp, sl,
              src_ids.data_ptr(), dst_ids.data_ptr(), n, _ptr(err_flag))
    return dst


def _page_state(block_table, seq_lens, ref_counts):
    i = _device(block_table, "block_table")
    R, max_blocks = block_table.shape
    _dense(block_table, i, "block_table", torch.int32, R, max_blocks)
    _dense(seq_lens, i, "seq_lens", torch.int32, R)
    pages = ref_counts.numel()
    _dense(ref_counts, i, "ref_counts", torch.int32, pages)
    return i, R, max_blocks, pages


def mla_kv_free(block_table, seq_lens, ref_counts, rows, *, block_size: int, err_flag=None,
                stream=None):
    """Give the pages of the rows [n] (int32) of block_table [R, max_blocks] back: their
    ref_counts [num_blocks] go down, their entries become -1 and their seq_lens 0."""
    i, R, max_blocks, pages = _page_state(block_table, seq_lens, ref_counts)
    n = rows.numel()
    _dense(rows, i, "rows", torch.int32, n)
    _err(err_flag, i)
    if n > 0:
        _call("mla_kv_free", i, stream, block_table.data_ptr(), seq_lens.data_ptr(),
              ref_counts.data_ptr(), rows.data_ptr(), n, R, pages, block_size, max_blocks, _ptr(err_flag))


def mla_kv_fork(kv_cache, block_table, seq_lens, ref_counts, parents, children, *,
                workspace=None, err_flag=None, stream=None):
    """Fork the sequences of rows parents [n] into the empty rows children [n]: full pages
    are shared (ref_counts), the last, partly filled page is copied in every layer of
    kv_cache ([num_blocks, bs, W] or [layers, num_blocks, bs, W]) to the lowest free page.
    workspace: a tensor of mla_kv_fork_workspace_size(n) bytes for this call alone (default:
    a new one; give one to keep when capturing into a graph)."""
    i, R, max_blocks, num_blocks = _page_state(block_table, seq_lens, ref_counts)
    layers, stride, pages, page_bytes, bs = _pools(kv_cache, "kv_cache")
    _on(kv_cache, i, "kv_cache")
    if pages != num_blocks:
        raise ValueError(f"ref_counts of {num_blocks} pages for a pool of {pages}")
    n = parents.numel()
    _dense(parents, i, "parents", torch.int32, n)
    _dense(children, i, "children", torch.int32, n)
    _err(err_flag, i)
    if n == 0:
        return
    if workspace is None:
        need = max(16, int(_ffi.lib().mla_kv_fork_workspace_size(n)))
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=block_table.device)
        else:
            with torch.cuda.stream(stream):     # freed in the order of the stream that uses it
                workspace = torch.empty(need, dtype=torch.uint8, device=block_table.device)
    else:
        _on(workspace, i, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _call("mla_kv_fork", i, stream, kv_cache.data_ptr(), stride, page_bytes, layers,
          block_table.data_ptr(), seq_lens.data_ptr(), ref_counts.data_ptr(), parents.data_ptr(),
          children.data_ptr(), n, R, num_blocks, bs, max_blocks, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), _ptr(err_flag))


def torch_dtype(name: str) -> torch.dtype:
    return _DT_TORCH[name]
