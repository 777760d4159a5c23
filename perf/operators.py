"""Measured cases of the cache operators: what a decode step does to the paged latent
cache besides the 16-bit and E4M3 attention.

    append  RMS norm of the latent, rotation of the RoPE key and of the queries' RoPE
            parts, and the rows' way into a paged cache of 16-bit, E4M3 or E2M1 values
    attend  the partial attention (per context shard, with its log-sum-exp) over a cache
            of E2M1 values: 4 bits each and an E4M3 scale for every 16
    fork    pages of sequences given back and sequences forked from others
            (full pages shared by reference count, the last, partly filled page copied)
    copy    pages of all layers copied from one pool to another by a list of ids

`run` computes each in its plain form with elementary torch operations, or, where `own` is
true, with the framework's calls.
"""
import math

import numpy as np
import torch

own = False

D_LAT, D_ROPE, D_QK = 512, 64, 576
E2M1_ROW = D_QK // 2 + D_QK // 16          # bytes of one cached token: codes, then scales
SCALE = 1.0 / math.sqrt(128 + 64)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence on one of eight ranks (16 heads): the smallest call of a
        # decode loop, where latency counts; the 16-bit cache
        dict(name="append_one", op="append", tokens=1, heads=16, kind="model", dtype="bf16", axes=1,
             interleaved=True, block_size=64),
        # a decode step of 32 sequences with every head on one GPU, E2M1 cache
        dict(name="append_decode", op="append", tokens=32, heads=128, kind="e2m1", dtype="bf16", axes=1,
             interleaved=True, block_size=64),
        # a chunk of prefill with image tokens (time, height, width positions) on one of eight
        # ranks, E2M1 cache
        dict(name="append_chunk", op="append", tokens=8192, heads=16, kind="e2m1", dtype="bf16", axes=3,
             interleaved=False, block_size=64),
        # a short history on one of eight ranks, one sequence: latency
        dict(name="attend_tiny", op="attend", batch=1, heads=16, q_len=1, shards=2, block_size=64,
             lo=256, hi=256, current=True, dtype="bf16"),
        # 32 sequences of 4096 tokens, all heads on one GPU
        dict(name="attend_dsv3", op="attend", batch=32, heads=128, q_len=1, shards=8, block_size=64,
             lo=4096, hi=4096, current=False, dtype="bf16"),
        # a ragged batch on one of eight ranks, fp16, pages of 32
        dict(name="attend_ragged", op="attend", batch=64, heads=16, q_len=1, shards=16, block_size=32,
             lo=512, hi=65536, current=False, dtype="fp16"),
        # two query tokens (multi-token prediction) over 32768 tokens with the current chunk
        dict(name="attend_mtp", op="attend", batch=8, heads=128, q_len=2, shards=8, block_size=32,
             lo=32768, hi=32768, current=True, dtype="bf16"),
        # very long histories on one of eight ranks
        dict(name="attend_verylong", op="attend", batch=16, heads=16, q_len=1, shards=16,
             block_size=64, lo=131072, hi=131072, current=False, dtype="bf16"),
        # a beam of four forked in one layer: latency
        dict(name="fork_beam", op="fork", forks=4, rows=8, layers=1, kind="e2m1", block_size=16,
             lo=100, hi=700),
        # 64 samples forked from prompts of up to 8192 tokens, four layers of a 16-bit cache
        dict(name="fork_samples", op="fork", forks=64, rows=96, layers=4, kind="model",
             block_size=64, lo=1024, hi=8192),
        # a few pages swapped out of one layer
        dict(name="copy_few", op="copy", pages=8, layers=1, pool=64, kind="e4m3", block_size=32),
        # the pages of long sequences packed into another pool, eight layers
        dict(name="copy_many", op="copy", pages=1024, layers=8, pool=2048, kind="e2m1", block_size=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "fork", "copy"])
    bs = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        heads = _log(rng, 1, 128)
        return dict(op=op, tokens=_log(rng, 1, min(8192, 131072 // heads)), heads=heads,
                    kind=rng.choice(["model", "e4m3", "e2m1", "e2m1"]), dtype=rng.choice(["bf16", "fp16"]),
                    axes=rng.choice([1, 1, 2, 3]), interleaved=rng.choice([True, False]), block_size=bs)
    if op == "attend":
        heads, q_len = rng.choice([8, 12, 16, 24, 32, 40, 64, 128, _log(rng, 1, 128)]), rng.choice([1, 1, 1, 2, 3, 4])
        hi = _log(rng, 40, 65536)
        lo = max(1, int(hi * rng.choice([0.02, 0.3, 1.0])))
        # at most 2^25 visible (row, token) pairs: below the largest listed case
        batch = _log(rng, 1, max(1, min(64, (1 << 25) // (hi * heads * q_len))))
        return dict(op=op, batch=batch, heads=heads, q_len=q_len, shards=rng.choice([1, 2, 3, 8, 16]), block_size=bs,
                    lo=lo, hi=hi, current=rng.choice([True, False]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "fork":
        forks, layers = _log(rng, 1, 64), _log(rng, 1, 4)
        return dict(op=op, forks=forks, rows=forks + _log(rng, 1, 32), layers=layers, kind=rng.choice(["model", "e4m3", "e2m1"]),
                    block_size=bs, lo=1, hi=_log(rng, 20, 4096))
    pages = _log(rng, 1, 512)
    return dict(op=op, pages=pages, layers=_log(rng, 1, 8), pool=2 * pages + _log(rng, 1, 100),
                kind=rng.choice(["model", "e4m3", "e2m1"]), block_size=min(bs, 128))


def _lengths(c):
    """History lengths: `lo`..`hi`, spread over their logarithm, the same for every seed
    (so that a case's work is known from the case alone)."""
    n = c.get("batch") or c["rows"]
    r = np.random.RandomState(n + c["hi"])
    return np.floor(np.exp(r.uniform(math.log(c["lo"]), math.log(c["hi"] + 0.999), n))).astype(np.int64)


def _row_bytes(kind):
    return {"model": 2 * D_QK, "e4m3": D_QK, "e2m1": E2M1_ROW}[kind]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _e2m1_round(x):
    """Magnitude codes of x >= 0: the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code."""
    return ((x > 0.25).to(torch.uint8) + (x >= 0.75) + (x > 1.25) + (x >= 1.75) + (x > 2.5) + (x >= 3.5) + (x > 5.0))


def _e4m3_round(x):
    """Nearest E4M3 values (ties to even, saturating at 448) of x in 64 bits."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _to_e2m1(x, kv_scale):
    """Codes [..., 288] and scales [..., 36] (bytes) of rows x [..., 576], and the values that
    they stand for.  scale = E4M3(max|x| / (6 kv_scale)) for each 16; code = E2M1(x / (scale kv_scale))."""
    g = x.reshape(*x.shape[:-1], D_QK // 16, 16)
    s = _e4m3_round(g.abs().amax(-1) / (6.0 * kv_scale))
    d = (s * kv_scale).unsqueeze(-1)
    m = _e2m1_round(torch.where(d > 0, g.abs() / torch.where(d > 0, d, 1.0), 0.0))
    code = (m | (torch.signbit(g).to(torch.uint8) << 3)).reshape(x.shape)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=x.dtype, device=x.device)
    value = torch.where(torch.signbit(g), -1.0, 1.0) * grid[m.long()] * d
    return packed, s.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8), value.reshape(x.shape)


def _e2m1_pages(n_blocks, bs, g, kv_scale):
    """A pool of E2M1 pages holding normed latents and keys: unit rows with channels of
    different strength."""
    pool = torch.empty(n_blocks, bs * E2M1_ROW, dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.3 * torch.randn(D_QK, generator=g, device="cuda"))
    step = max(1, (1 << 17) // bs)
    for a in range(0, n_blocks, step):
        n = min(step, n_blocks - a)
        codes, scales, _ = _to_e2m1(torch.randn(n, bs, D_QK, generator=g, device="cuda") * gain, kv_scale)
        pool[a:a + n, :bs * D_QK // 2] = codes.reshape(n, -1)
        pool[a:a + n, bs * D_QK // 2:] = scales.reshape(n, -1)
    return pool.view(n_blocks, bs, E2M1_ROW)


def _cos_sin(max_pos):
    """cos and sin of position * 10000^(-i/32), computed in 64 bits: [max_pos, 64]."""
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _sections(axes):
    return {1: [32], 2: [16, 16], 3: [8, 12, 12]}[axes]


def prepare(case, seed):
    c, g = case, _gen(seed)
    dev = "cuda"
    if c["op"] == "append":
        T, H, bs, dt = c["tokens"], c["heads"], c["block_size"], DT[c["dtype"]]
        blocks = -(-T // bs) + 3
        slots = torch.randperm(blocks * bs, generator=g, device=dev)[:T].to(torch.int32)
        if T > 4:
            slots[T // 2] = -1                     # a padded token: stored nowhere
        pool = torch.zeros(blocks, bs, E2M1_ROW if c["kind"] == "e2m1" else D_QK, device=dev,
                           dtype=dt if c["kind"] == "model" else torch.uint8)
        kv_a = torch.randn(T, D_QK, generator=g, device=dev) * torch.exp(
            0.5 * torch.randn(D_QK, generator=g, device=dev))
        q = torch.randn(T, H, 192, generator=g, device=dev)
        kv_a, q = kv_a.to(dt), q.to(dt)
        return dict(case=c, c_kv=kv_a[:, :D_LAT], k_pe=kv_a[:, D_LAT:], q_pe=q[:, :, 128:],
                    weight=(1 + 0.2 * torch.randn(D_LAT, generator=g, device=dev)).to(dt), pool=pool, slots=slots,
                    positions=torch.randint(0, 131072, (c["axes"], T), generator=g, device=dev, dtype=torch.int32),
                    cos_sin=_cos_sin(131072), kv_scale=2.0 ** -4, err=torch.zeros(1, dtype=torch.int32, device=dev))
    if c["op"] == "attend":
        B, H, q, bs, dt = c["batch"], c["heads"], c["q_len"], c["block_size"], DT[c["dtype"]]
        lens = _lengths(c)
        per = -(-lens // bs)
        perm = torch.randperm(int(per.sum()), generator=g, device=dev).to(torch.int32)
        where = np.full((B, int(per.max())), -1, np.int64)
        for b, (a, n) in enumerate(zip(np.cumsum(per) - per, per)):
            where[b, :n] = a + np.arange(n)
        where = torch.from_numpy(where).to(dev)
        table = torch.where(where >= 0, perm[where.clamp(min=0)], -1).to(torch.int32)
        scale = 2.0 ** -4
        cur = torch.randn(B, q, D_QK, generator=g, device=dev).to(dt) if c["current"] else None
        return dict(case=c, pool=_e2m1_pages(int(per.sum()), bs, g, scale), kv_scale=scale, table=table, kv_cur=cur,
                    lens=torch.from_numpy(lens.astype(np.int32)).to(dev),
                    q_abs=torch.randn(B, q, H, D_LAT, generator=g, device=dev).to(dt),
                    q_pe=torch.randn(B, q, H, D_ROPE, generator=g, device=dev).to(dt),
                    err=torch.zeros(1, dtype=torch.int32, device=dev))
    bs, layers = c["block_size"], c["layers"]
    row = _row_bytes(c["kind"]) // (2 if c["kind"] == "model" else 1)

    def pool(n):
        x = torch.randint(0, 256, (layers, n, bs * _row_bytes(c["kind"])), generator=g, device=dev, dtype=torch.uint8)
        if c["kind"] == "model":
            x.view(torch.int16).bitwise_and_(-0x2001)      # any bits but those of infinities and NaN
        return (x.view(torch.bfloat16) if c["kind"] == "model" else x).view(layers, n, bs, row)

    if c["op"] == "copy":
        ids = torch.randperm(c["pool"], generator=g, device=dev)[:c["pages"]].to(torch.int32)
        to = torch.randperm(c["pages"] + 5, generator=g, device=dev)[:c["pages"]].to(torch.int32)
        return dict(case=c, src=pool(c["pool"]), dst=pool(c["pages"] + 5), src_ids=ids, dst_ids=to,
                    err=torch.zeros(1, dtype=torch.int32, device=dev))
    # fork: rows 0..live-1 are sequences, the other `forks` rows their forks of the step before
    R, n = c["rows"], c["forks"]
    live = R - n
    lens = _lengths(c)
    lens[live:] = lens[np.random.RandomState(n).randint(0, live, n)]
    per = -(-lens // bs)
    used = int(per.sum())
    blocks = used + n + 8
    perm = torch.randperm(blocks, generator=g, device=dev).cpu().numpy()
    table = np.full((R, int(per.max()) + 2), -1, np.int32)
    for r, (a, k) in enumerate(zip(np.cumsum(per) - per, per)):
        table[r, :k] = perm[a:a + k]
    refs = np.zeros(blocks, np.int32)
    refs[perm[:used]] = 1
    rows = np.arange(live, R, dtype=np.int32)
    parents = torch.randint(0, live, (n,), generator=g, device=dev, dtype=torch.int32)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    return dict(case=c, pool=pool(blocks), table=to(table), lens=to(lens.astype(np.int32)), refs=to(refs),
                parents=parents, children=to(rows), err=torch.zeros(1, dtype=torch.int32, device=dev))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _append, "attend": _attend, "fork": _fork, "copy": _copy}[state["case"]["op"]](state)


def _append(s):
    c = s["case"]
    kind, dt = c["kind"], DT[c["dtype"]]
    if own:
        from mla_decode_attention_kv_gb300 import api
        q_out, kv_out = api.mla_kv_append(
            s["c_kv"], s["k_pe"], s["pool"], s["slots"], s["positions"], s["cos_sin"], norm_weight=s["weight"],
            eps=1e-6, q_pe=s["q_pe"], kv_out="new", kv_scale=None if kind == "model" else s["kv_scale"],
            interleaved=c["interleaved"], sections=_sections(c["axes"]), err_flag=s["err"])
        return _stored(kind, q_out, kv_out, s["pool"])
    # in 64 bits: what is stored in 8 or 4 bits lies next to borders
    x = s["c_kv"].double()
    lat = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].double()
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=x.device),
                                   torch.tensor(_sections(c["axes"]), device=x.device))     # of each pair
    cs = s["cos_sin"].double()
    pos = s["positions"].long()[axis].T                                                     # [T, 32]
    pair = torch.arange(32, device=x.device)
    cos, sin = cs[pos, pair], cs[pos, pair + 32]

    def rotate(v, co, si):
        if c["interleaved"]:
            a, b = v[..., 0::2], v[..., 1::2]
            return torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
        a, b = v[..., :32], v[..., 32:]
        return torch.cat([a * co - b * si, a * si + b * co], -1)

    row = torch.cat([lat, rotate(s["k_pe"].double(), cos, sin)], -1)
    q_out = rotate(s["q_pe"].float(), cos.float()[:, None], sin.float()[:, None]).to(dt)
    at = s["slots"] >= 0
    slot = s["slots"][at].long()
    pool = s["pool"]
    if kind == "model":
        kv_out = row.to(dt)
        pool.view(-1, D_QK)[slot] = kv_out[at]
    elif kind == "e4m3":
        kv_out = _e4m3_round(row / s["kv_scale"]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        pool.view(-1, D_QK)[slot] = kv_out[at]
    else:
        codes, scales, value = _to_e2m1(row, s["kv_scale"])
        kv_out = value.to(dt)
        bs = c["block_size"]
        pages = pool.view(pool.shape[0], -1)
        pages[:, :bs * 288].unflatten(1, (bs, 288))[slot // bs, slot % bs] = codes[at]
        pages[:, bs * 288:].unflatten(1, (bs, 36))[slot // bs, slot % bs] = scales[at]
    return _stored(kind, q_out, kv_out, pool)


def _stored(kind, q_out, kv_out, pool):
    """The outputs: E4M3 bytes as the numbers that they are.  E2M1 rows come back as the values
    they stand for in kv_out, and the pool's bytes with them."""
    if kind == "e4m3":
        return {"q": q_out, "kv": kv_out.view(torch.float8_e4m3fn), "pool": pool.view(torch.float8_e4m3fn)}
    return {"q": q_out, "kv": kv_out, "pool": pool}


def _attend(s):
    c = s["case"]
    if own:
        from mla_decode_attention_kv_gb300 import api
        o, lse = api.mla_dcp_decode_partial(s["q_abs"], s["q_pe"], s["pool"], s["table"], s["lens"], c["shards"],
                                            kv_cur=s["kv_cur"], kv_scale=s["kv_scale"], err_flag=s["err"])
        return {"o": o, "lse": lse}
    B, H, n_q, S, bs = c["batch"], c["heads"], c["q_len"], c["shards"], c["block_size"]
    dev, dt = s["pool"].device, DT[c["dtype"]]
    pages = s["pool"].view(s["pool"].shape[0], -1)
    codes = pages[:, :bs * 288].unflatten(1, (bs, 288))
    scales = pages[:, bs * 288:].unflatten(1, (bs, 36))
    lens = s["lens"].long()
    width = bs * -(-lens // (S * bs))                                                     # tokens of a shard
    most = int(bs * -(-c["hi"] // (S * bs)))
    k = torch.arange(most, device=dev)
    start = torch.arange(S, device=dev)[None, :] * width[:, None]                         # [B, S]
    tok = start[..., None] + k                                                            # [B, S, most]
    seen = (k < width[:, None, None]) & (tok < lens[:, None, None])
    tok = torch.where(seen, tok, 0)
    page = torch.gather(s["table"].long(), 1, (tok // bs).flatten(1)).view_as(tok).clamp(min=0)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=dev)
    two = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], 1)                   # both values of a byte
    kv = two[codes[page, tok % bs].int()].flatten(-2)                                     # [B, S, most, 576]
    kv.unflatten(-1, (36, 16)).mul_(
        (scales[page, tok % bs].view(torch.float8_e4m3fn).float() * s["kv_scale"]).unsqueeze(-1))
    q = torch.cat([s["q_abs"], s["q_pe"]], -1).float().flatten(1, 2)                      # [B, q H, 576]

    def part(kv, seen):
        logits = SCALE * torch.matmul(q[:, None], kv.transpose(-1, -2))                   # [B, S, q H, n]
        logits = logits.masked_fill(~seen, float("-inf"))
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
        z = p.sum(-1, keepdim=True)
        lse = (torch.log(z) + top).squeeze(-1)
        return torch.matmul(p, kv[..., :D_LAT]) / torch.where(z > 0, z, 1.0), lse

    o, lse = part(kv, seen[:, :, None])
    if s["kv_cur"] is not None:
        i = torch.arange(n_q, device=dev).repeat_interleave(H)
        o1, lse1 = part(s["kv_cur"].float()[:, None], (torch.arange(n_q, device=dev) <= i[:, None])[None, None])
        o, lse = torch.cat([o, o1], 1), torch.cat([lse, lse1], 1)
    P = o.shape[1]
    return {"o": o.to(dt).view(B, P, n_q, H, D_LAT).transpose(1, 2).contiguous(),
            "lse": lse.view(B, P, n_q, H).transpose(1, 2).contiguous()}


def _fork(s):
    c = s["case"]
    bs = c["block_size"]
    table, lens, refs, pool = s["table"], s["lens"], s["refs"], s["pool"]
    kids, parents = s["children"].long(), s["parents"].long()
    if own:
        from mla_decode_attention_kv_gb300 import api
        api.mla_kv_free(table, lens, refs, s["children"], block_size=bs, err_flag=s["err"])
        api.mla_kv_fork(pool, table, lens, refs, s["parents"], s["children"], err_flag=s["err"])
        return {"table": table, "lens": lens, "refs": refs, "pool": pool}
    # give back what the forked rows hold
    col = torch.arange(table.shape[1], device=table.device)
    held = col < (-(-lens[kids] // bs))[:, None]
    refs.scatter_add_(0, table[kids].clamp(min=0).long().flatten(), -held.int().flatten())
    table[kids] = -1
    lens[kids] = 0
    # share the full pages, take the lowest free pages for the copies of the last ones
    n = lens[parents].long()
    old = table[parents]
    full, some = n // bs, n % bs > 0
    share = col < full[:, None]
    fresh = torch.sort(refs > 0, stable=True).indices[:c["forks"]]
    fresh = fresh[(torch.cumsum(some, 0) - 1).clamp(min=0)]
    new = torch.where(share, old, -1)
    last = full.clamp(max=table.shape[1] - 1)[:, None]
    new.scatter_(1, last, torch.where(some, fresh.int(), torch.gather(new, 1, last)[:, 0])[:, None])
    refs.scatter_add_(0, old.clamp(min=0).long().flatten(), share.int().flatten())
    refs[fresh[some]] = 1
    pool[:, fresh[some]] = pool[:, torch.gather(old, 1, last)[:, 0].long()[some]]
    table[kids] = new
    lens[kids] = n.int()
    return {"table": table, "lens": lens, "refs": refs, "pool": pool}


def _copy(s):
    if own:
        from mla_decode_attention_kv_gb300 import api
        api.mla_kv_copy_pages(s["src"], s["dst"], s["src_ids"], s["dst_ids"], err_flag=s["err"])
    else:
        s["dst"][:, s["dst_ids"].long()] = s["src"][:, s["src_ids"].long()]
    return {"pool": s["dst"]}


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "append":
        T, H = c["tokens"], c["heads"]
        out = {"model": 2 * D_QK, "e4m3": D_QK, "e2m1": 2 * D_QK}[c["kind"]]     # kv_out
        per = 2 * D_QK + 2 * 2 * H * D_ROPE + out + _row_bytes(c["kind"]) + 4 * c["axes"] + 4 + 256
        return {"bytes": T * per + 2 * D_LAT, "flops": T * (6 * D_LAT + 6 * 32 * (H + 1))}
    if c["op"] == "attend":
        lens = _lengths(c)
        rows = c["batch"] * c["q_len"] * c["heads"]
        parts = c["shards"] + (1 if c["current"] else 0)
        kv = int(lens.sum()) * E2M1_ROW + int((-(-lens // c["block_size"])).sum()) * 4
        seen = int(lens.sum()) * c["q_len"]
        if c["current"]:
            kv += c["batch"] * c["q_len"] * 2 * D_QK
            seen += c["batch"] * c["q_len"] * (c["q_len"] + 1) // 2
        return {"bytes": kv + rows * 2 * D_QK + rows * parts * (2 * D_LAT + 4),
                "flops": 2 * c["heads"] * (D_QK + D_LAT) * seen}
    page = c["block_size"] * _row_bytes(c["kind"]) * c["layers"]
    if c["op"] == "copy":
        return {"bytes": c["pages"] * (2 * page + 8), "flops": 0}
    # fork: which parents are drawn varies with the seed; the mean number of copies and of pages
    live = c["rows"] - c["forks"]
    lens = _lengths(c)[:live]
    some = float((lens % c["block_size"] > 0).mean())
    pages = float((-(-lens // c["block_size"])).mean())
    return {"bytes": int(c["forks"] * (some * 2 * page + 7 * 4 * pages)) + 64, "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def _decode_e2m1(nib):
    """Values of 4-bit codes from the format: sign, two exponent bits (bias 1), one mantissa bit."""
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, e.double() - 1))
    return torch.where((nib >> 3) == 1, -mag, mag)


def _decode_e4m3(b):
    """Values of E4M3 bytes from the format: sign, four exponent bits (bias 7), three mantissa bits."""
    b = b.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, e.double() - 10))
    return torch.where(b >> 7 == 1, -mag, mag)


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "copy"):
        return None                       # whole numbers and bytes that only move
    s = prepare(case, seed)
    if c["op"] == "append":
        T = c["tokens"]
        c_kv, k_pe, q_pe = s["c_kv"].double(), s["k_pe"].double(), s["q_pe"].double()
        ms = (c_kv * c_kv).sum(1) / D_LAT
        lat = s["weight"].double() * c_kv / torch.sqrt(ms + 1e-6)[:, None]
        which = []
        for a, n in enumerate(_sections(c["axes"])):
            which += [a] * n
        rot = torch.empty(T, 32, dtype=torch.complex128, device="cuda")
        for i, a in enumerate(which):
            t = s["cos_sin"][s["positions"][a].long()].double()
            rot[:, i] = torch.complex(t[:, i], t[:, 32 + i])

        def turn(v, w):
            if c["interleaved"]:
                z = torch.view_as_complex(v.contiguous().unflatten(-1, (32, 2))) * w
                return torch.view_as_real(z).flatten(-2)
            z = torch.complex(v[..., :32], v[..., 32:]) * w
            return torch.cat([z.real, z.imag], -1)

        row = torch.cat([lat, turn(k_pe, rot)], 1)
        q = turn(q_pe, rot[:, None])
        if c["kind"] == "model":
            pool = s["pool"].double().view(-1, D_QK)
            keep = (s["slots"] >= 0).nonzero()[:, 0]
            pool[s["slots"][keep].long()] = row[keep]
            return {"q": q, "kv": row, "pool": pool.view(s["pool"].shape)}
        # what rounding to 8 or 4 bits makes of a row is not a number that has a closer one
        return {"q": q, "kv": None, "pool": None}
    B, H, n_q, S, bs = c["batch"], c["heads"], c["q_len"], c["shards"], c["block_size"]
    P = S + (1 if c["current"] else 0)
    o = torch.zeros(B, n_q, P, H, D_LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n_q, P, H), float("-inf"), dtype=torch.float64, device="cuda")
    q = torch.cat([s["q_abs"], s["q_pe"]], -1).double()

    def fill(b, i, p, kv):
        z = (q[b, i] @ kv.T) * SCALE                                      # [H, n]
        lse[b, i, p] = torch.logsumexp(z, 1)
        o[b, i, p] = torch.exp(z - lse[b, i, p][:, None]) @ kv[:, :D_LAT]

    for b in range(B):
        L = int(s["lens"][b])
        ids = s["table"][b, :-(-L // bs)].long()
        raw = s["pool"].view(s["pool"].shape[0], -1)[ids]
        code, sc = raw[:, :bs * 288].reshape(-1, 288), raw[:, bs * 288:].reshape(-1, 36)
        val = torch.stack([_decode_e2m1(code.int() & 15), _decode_e2m1(code.int() >> 4)], -1).flatten(1)
        val = (val.unflatten(1, (36, 16)) * (_decode_e4m3(sc) * s["kv_scale"])[:, :, None]).flatten(1)[:L]
        w = bs * -(-L // (S * bs))
        for p in range(S):
            kv = val[p * w:min(L, (p + 1) * w)]
            for i in range(n_q):
                if kv.shape[0]:
                    fill(b, i, p, kv)
        for i in range(n_q if c["current"] else 0):
            fill(b, i, S, s["kv_cur"][b, :i + 1].double())
    return {"o": o, "lse": lse}
