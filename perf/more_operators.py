"""Workloads of dense attention over a paged 8-bit cache whose blocks share a
scale, and of what feeds it: the norms and rotations of the heads' queries and
keys, and the quantising write into that cache.

Each case is one call of one operator on inputs as a serving loop has them.
With ``own`` false ``run`` computes the operator from elementary torch
operations; with ``own`` true it calls this package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request: index keys' layer norm, half the head rotated in neighbouring pairs
        {"name": "rope_one_token", "op": "rope", "tokens": 1, "heads": 32, "kv_heads": 1, "dim": 128, "rot": 64,
         "start": 0, "norm": "layer", "interleaved": True, "type": "bf16", "far": 131072},
        # a speculative decode step of 16 requests of 6 rows, grouped heads, far positions
        {"name": "rope_verify_96", "op": "rope", "tokens": 96, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "start": 0, "norm": "rms", "interleaved": False, "type": "bf16", "far": 131072},
        # an odd chunk with three key heads; the rotated part stands last in the head
        {"name": "rope_odd_d64", "op": "rope", "tokens": 4099, "heads": 21, "kv_heads": 3, "dim": 64, "rot": 48,
         "start": 16, "norm": "rms", "interleaved": False, "type": "f32", "far": 16384},
        # a large prompt chunk
        {"name": "rope_prompt_16384", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "start": 0, "norm": "rms", "interleaved": False, "type": "bf16", "far": 32768},
        # the new tokens of a speculative decode step
        {"name": "store_verify_96", "op": "store", "requests": 16, "new": 6, "heads": 8, "dim": 128, "block": 64,
         "type": "bf16"},
        # prompt chunks of odd lengths, small blocks, single precision
        {"name": "store_odd_d64", "op": "store", "requests": 7, "new": 509, "heads": 3, "dim": 64, "block": 16,
         "type": "f32"},
        # a large prompt chunk
        {"name": "store_prompt_16384", "op": "store", "requests": 8, "new": 2048, "heads": 8, "dim": 128, "block": 64,
         "type": "bf16"},
        # one request, one token, short context: latency
        {"name": "attn_one_token", "op": "attn", "requests": 1, "new": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 64, "length": 1024, "window": 0},
        # speculative verify: 16 requests of 6 rows over long contexts, one key head
        {"name": "attn_verify_131072", "op": "attn", "requests": 16, "new": 6, "heads": 32, "kv_heads": 1, "dim": 128,
         "block": 64, "length": 131072, "window": 0},
        # a large decode batch with grouped heads
        {"name": "attn_decode_32768", "op": "attn", "requests": 32, "new": 1, "heads": 64, "kv_heads": 8, "dim": 128,
         "block": 128, "length": 32768, "window": 0},
        # prompt chunks of four requests
        {"name": "attn_prompt_4x2048", "op": "attn", "requests": 4, "new": 2048, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 64, "length": 8192, "window": 0},
        # odd sizes: three key heads of seven heads, small blocks, a sliding window
        {"name": "attn_odd_window_d64", "op": "attn", "requests": 5, "new": 259, "heads": 21, "kv_heads": 3,
         "dim": 64, "block": 16, "length": 4095, "window": 1000},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "store", "attn", "attn"])
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    dim = rng.choice([64, 128])
    if op == "rope":
        heads = kv_heads * rng.choice([1, 2, 5, 7, 8, 16])
        kind = rng.choice(["bf16", "f16", "f32"])
        interleaved = rng.random() < 0.4
        rot = rng.randint(1, dim // 8) * 8 if interleaved else rng.randint(1, dim // 16) * 16
        most = 16384 * 40 * 128 // ((heads + kv_heads) * dim * (2 if kind == "f32" else 1))
        return {"op": op, "tokens": _log_int(rng, 1, min(most, 65536)), "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "rot": rot, "start": rng.randint(0, (dim - rot) // 8) * 8,
                "norm": rng.choice(["none", "rms", "rms", "layer"]), "interleaved": interleaved, "type": kind,
                "far": _log_int(rng, 1000, 1 << 20)}
    block = rng.choice([16, 32, 64, 128])
    if op == "store":
        kind = rng.choice(["bf16", "f16", "f32"])
        most = 16384 * 8 * 128 // (kv_heads * dim * (2 if kind == "f32" else 1))
        requests = _log_int(rng, 1, 256)
        return {"op": op, "requests": requests, "new": _log_int(rng, 1, max(1, min(most, 32768) // requests)),
                "heads": kv_heads, "dim": dim, "block": block, "type": kind}
    group = rng.choice([1, 2, 5, 7, 8, 16, 32])
    if rng.random() < 0.5:  # decode rows
        requests, new = _log_int(rng, 1, 64), rng.randint(1, 6)
        length = _log_int(rng, 16, max(64, min(131072, 32 * 8 * 32768 // (requests * kv_heads))))
    else:  # prompt chunks
        requests, new = rng.randint(1, 6), _log_int(rng, 7, 2048)
        length = new + _log_int(rng, 1, 6144)
    # no more scores than the largest listed case has
    group = max(1, min(group, 4 * 2048 * 32 * 8192 // (requests * new * length * kv_heads)))
    return {"op": op, "requests": requests, "new": new, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
            "block": block, "length": length, "window": rng.choice([0, 0, _log_int(rng, 1, 4096)])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def page_bytes(block, dim):
    """Bytes of one head's page: the e4m3 key and value row of each token, then
    the keys' and the values' f32 scale, then 8 bytes without meaning."""
    return block * 2 * dim + 16


def _code_view(cache, block, dim):
    """cache [..., page] u8 -> its e4m3 bytes [..., block, 2, dim]."""
    return cache[..., : block * 2 * dim].unflatten(-1, (block, 2, dim))


def _scale_view(cache, block, dim):
    """cache [..., page] u8 -> its scales [..., 2] f32."""
    return cache[..., block * 2 * dim: block * 2 * dim + 8].view(torch.float32)


def _fill_cache(cache, g, block, dim):
    """Keys and values ~ N(0, 1) with a scale for each page."""
    codes, scales = _code_view(cache, block, dim), _scale_view(cache, block, dim)
    rows = max(1, (1 << 28) // codes[0].numel())
    for at in range(0, cache.shape[0], rows):  # in parts: the f32 draws of a whole cache need not fit
        x = torch.randn(codes[at: at + rows].shape, generator=g, device=DEV)
        s = x.abs().amax((-3, -1)) / E4M3_MAX
        codes[at: at + rows] = (x / s[..., None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(
            torch.uint8)
        scales[at: at + rows] = s


def _prepare_rope(c, seed):
    g = _gen(seed)
    T, D, kind = c["tokens"], c["dim"], _TYPES[c["type"]]
    x = [(3 * torch.randn((T, h, D), generator=g, device=DEV)).to(kind) for h in (c["heads"], c["kv_heads"])]
    positions = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    if T > 8:  # rows that pad the step
        positions[-3:] = -1
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    s = {"q": x[0], "k": x[1], "positions": positions, "inv_freq": (10000.0 ** (-2 * i / c["rot"])).float(),
         "out_q": torch.zeros_like(x[0]), "out_k": torch.zeros_like(x[1])}
    for n in ("q_weight", "k_weight", "q_bias", "k_bias"):
        v = 0.2 * torch.randn(D, generator=g, device=DEV) + (1.0 if "weight" in n else 0.0)
        s[n] = v if c["norm"] == "layer" or (c["norm"] == "rms" and "weight" in n) else None
    return s


def _prepare_store(c, seed):
    g = _gen(seed)
    B, H, D, bs = c["requests"], c["heads"], c["dim"], c["block"]
    new = torch.randint((c["new"] + 1) // 2, c["new"] + 1, (B,), generator=g, device=DEV)
    new[0] = c["new"]
    held = torch.randint(0, bs, (B,), generator=g, device=DEV)  # tokens that the request's last block holds
    blocks = B * (-(-(c["new"] + bs) // bs)) + 8
    tables = torch.randperm(blocks, generator=g, device=DEV)[: blocks - 8].view(B, -1)
    T = B * c["new"]
    cu = new.cumsum(0)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu, t, right=True).clamp(max=B - 1)
    pos = held[b] + t - (cu[b] - new[b])
    slots = torch.where(t < cu[-1], tables[b, (pos // bs).clamp(max=tables.shape[1] - 1)] * bs + pos % bs,
                        torch.full_like(t, -1)).int()
    cache = torch.zeros((blocks, H, page_bytes(bs, D)), dtype=torch.uint8, device=DEV)
    _fill_cache(cache, g, bs, D)
    x = [(torch.randn((T, H, D), generator=g, device=DEV)
          * torch.exp(0.5 * torch.randn((T, H, 1), generator=g, device=DEV))).to(_TYPES[c["type"]]) for _ in range(2)]
    return {"k": x[0], "v": x[1], "slot_mapping": slots, "kv_cache": cache}


def _prepare_attn(c, seed):
    g = _gen(seed)
    B, H, HK, D, bs, L = (c[x] for x in ("requests", "heads", "kv_heads", "dim", "block", "length"))
    n = min(c["new"], L)
    if n <= 8:  # decode: every request has the same rows
        new = torch.full((B,), n, dtype=torch.int64, device=DEV)
    else:
        new = torch.randint((n + 1) // 2, n + 1, (B,), generator=g, device=DEV)
        new[0] = n
    lens = torch.maximum(L - (torch.rand(B, generator=g, device=DEV) * 0.3 * L).long(), new)
    lens[0] = L
    max_blocks = -(-L // bs)
    blocks = B * max_blocks + 8
    cache = torch.zeros((blocks, HK, page_bytes(bs, D)), dtype=torch.uint8, device=DEV)
    _fill_cache(cache, g, bs, D)
    tables = torch.randperm(blocks, generator=g, device=DEV)[: B * max_blocks].int().view(B, max_blocks)
    q = torch.randn((B * n, H, D), generator=g, device=DEV).to(torch.bfloat16)
    return {"q": q, "kv_cache": cache, "block_tables": tables, "context_lens": lens.int(),
            "cu_new_lens": torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), new.cumsum(0)]).int(),
            "scale": 1.0 / math.sqrt(D), "out": torch.zeros_like(q),
            "lse": torch.zeros((B * n, H), dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    return {"op": case["op"], "case": dict(case),
            **{"rope": _prepare_rope, "store": _prepare_store, "attn": _prepare_attn}[case["op"]](case, seed)}


# -------------------------------------------------------------- plain forms
def _plain_norm_rope(c, x, weight, bias, cos, sin):
    y = x.float()
    if c["norm"] == "rms":
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    if c["norm"] == "layer":
        y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    lo, hi = c["start"], c["start"] + c["rot"]
    r = y[..., lo:hi]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([p, q], -1).flatten(-2) if c["interleaved"] else torch.cat([p, q], -1)
    return torch.cat([y[..., :lo], r, y[..., hi:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    live = (s["positions"] >= 0)[:, None, None]
    return {n: torch.where(live, _plain_norm_rope(c, s[n[-1]], s[n[-1] + "_weight"], s[n[-1] + "_bias"], cos, sin), s[n])
            for n in ("out_q", "out_k")}


def _stored(s):
    """The cache's content as the values it stands for."""
    c = s["case"]
    return {"codes": _code_view(s["kv_cache"].view(torch.float8_e4m3fn), c["block"], c["dim"]),
            "scales": _scale_view(s["kv_cache"], c["block"], c["dim"])}


def _plain_store(s):
    c = s["case"]
    bs, D, H = c["block"], c["dim"], c["heads"]
    codes, scales = _code_view(s["kv_cache"], bs, D), _scale_view(s["kv_cache"], bs, D)
    blocks = codes.shape[0]
    keep = s["slot_mapping"] >= 0
    slot = s["slot_mapping"][keep].long()
    blk, off = slot // bs, slot % bs
    x = torch.stack([s["k"][keep], s["v"][keep]], 2).float()  # [n, H, 2, D]
    # a block's first new token and the largest value of its new tokens
    first = torch.full((blocks,), bs, dtype=torch.int64, device=DEV).scatter_reduce(0, blk, off, "amin")
    top = torch.zeros((blocks, H, 2), device=DEV).scatter_reduce(
        0, blk[:, None, None].expand(-1, H, 2), x.abs().amax(-1), "amax")
    need = top / E4M3_MAX
    held = (first > 0) & (first < bs)  # blocks that hold tokens and get more
    old = scales.clone()
    (mn, en), (mo, eo) = torch.frexp(need), torch.frexp(old)
    grow = ((en - eo) + (mn > mo)).clamp(min=0)  # old * 2^grow is the first one at or above need
    grow = torch.where((need > 0) & (old > 0) & held[:, None, None], grow, torch.zeros_like(grow))
    fresh = (first == 0)[:, None, None] | ((old == 0) & held[:, None, None])
    scales.copy_(torch.where(fresh, need, torch.ldexp(old, grow)))
    again = held[:, None, None, None] & (torch.arange(bs, device=DEV)[:, None] < first[:, None, None, None])
    shifted = torch.ldexp(codes.view(torch.float8_e4m3fn).float(), -grow[:, :, None, :, None])
    codes.copy_(torch.where((again & (grow > 0)[:, :, None])[..., None], shifted.to(torch.float8_e4m3fn).view(torch.uint8),
                            codes))
    sc = scales[blk][..., None]
    y = torch.where(sc == 0, torch.zeros_like(x), x / sc).clamp(-E4M3_MAX, E4M3_MAX)
    codes[blk, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return _stored(s)


def _plain_attn(s):
    c = s["case"]
    bs, D, HK, L = c["block"], c["dim"], c["kv_heads"], c["length"]
    G = c["heads"] // HK
    tables, cu = s["block_tables"].long(), s["cu_new_lens"].long()
    ctx = s["context_lens"].long()
    B = ctx.shape[0]
    new = cu[1:] - cu[:-1]
    N = min(c["new"], L)
    codes = _code_view(s["kv_cache"], bs, D)[tables].view(torch.float8_e4m3fn)  # [B, blocks, HK, bs, 2, D]
    kv = codes.float() * _scale_view(s["kv_cache"], bs, D)[tables][:, :, :, None, :, None]
    del codes
    kv = kv.permute(4, 0, 2, 1, 3, 5).reshape(2, B, HK, -1, D)[:, :, :, :L]
    n = torch.arange(N, device=DEV)
    row = (cu[:-1, None] + n).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, N, HK, G, D).permute(0, 2, 1, 3, 4).reshape(B, HK, N * G, D)
    score = torch.matmul(q, kv[0].transpose(-1, -2)).view(B, HK, N, G, L) * s["scale"]
    pos = (ctx - new)[:, None] + n
    j = torch.arange(L, device=DEV)
    seen = (j <= pos[..., None]) & ((j > pos[..., None] - c["window"]) if c["window"] else True)
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del score
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, HK, N * G, L), kv[1]).view(B, HK, N, G, D) / torch.where(
        total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    real = n < new[:, None]
    at = row[real]
    s["out"][at] = out.permute(0, 2, 1, 3, 4).reshape(B, N, HK * G, D)[real].to(s["out"].dtype)
    s["lse"][at] = lse.permute(0, 2, 1, 3).reshape(B, N, HK * G)[real]
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------- runs
def run(state):
    s = state
    if own:
        import sparse_attention_fp8_gb300 as fp8idx
        c = s["case"]
        if s["op"] == "rope":
            fp8idx.head_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["out_q"], s["out_k"],
                                  norm=c["norm"], q_weight=s["q_weight"], q_bias=s["q_bias"],
                                  k_weight=s["k_weight"], k_bias=s["k_bias"], eps=1e-6,
                                  interleaved=c["interleaved"], rot_start=c["start"])
            return {"out_q": s["out_q"], "out_k": s["out_k"]}
        if s["op"] == "store":
            fp8idx.fp8_paged_block_store(s["k"], s["v"], s["slot_mapping"], s["kv_cache"])
            return _stored(s)
        if "workspace" not in s:  # a serving loop keeps one
            s["workspace"] = torch.empty(fp8idx.paged_block_attn_workspace(c["dim"]), dtype=torch.uint8, device=DEV)
        fp8idx.fp8_paged_block_attn(s["q"], s["kv_cache"], s["block_tables"], s["context_lens"], s["cu_new_lens"],
                                    s["scale"], s["out"], lse=s["lse"], window=c["window"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"rope": _plain_rope, "store": _plain_store, "attn": _plain_attn}[s["op"]](s)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        size = 4 if c["type"] == "f32" else 2
        n = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * n * size + 4 * c["tokens"] + 2 * c["rot"], "flops": 8 * n}
    if c["op"] == "store":
        # ragged chunks: three quarters of the rows are tokens, the others pad the step
        tokens = c["requests"] * (c["new"] * 3 + 1) // 4
        size = 4 if c["type"] == "f32" else 2
        n = tokens * c["heads"] * 2 * c["dim"]
        blocks = c["requests"] + tokens // c["block"]
        return {"bytes": n * (size + 1) + 16 * blocks * c["heads"] + 4 * c["requests"] * c["new"], "flops": 2 * n}
    new, L = min(c["new"], c["length"]), c["length"]
    mean_new = new if new <= 8 else (3 * new + 1) / 4
    mean_len = max(mean_new, L * (0.85 + 0.15 / c["requests"]))
    reach = mean_len - (mean_new - 1) / 2  # positions up to a row's own, on average
    seen = min(reach, c["window"]) if c["window"] else reach
    read = min(mean_len, c["window"] + mean_new) if c["window"] else mean_len
    rows = c["requests"] * mean_new
    kv = c["requests"] * read * c["kv_heads"] * (2 * c["dim"] + 8 / c["block"])
    return {"bytes": int(kv + rows * c["heads"] * (4 * c["dim"] + 4)),
            "flops": int(4 * rows * c["heads"] * seen * c["dim"])}


# -------------------------------------------------------------------- exact
def _exact_rope(c, s):
    out = {}
    phase = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(phase), phase)[:, None]
    lo, hi, half = c["start"], c["start"] + c["rot"], c["rot"] // 2
    for n in ("q", "k"):
        x = s[n].double()
        if c["norm"] == "layer":
            x = x - x.mean(-1, keepdim=True)
        if c["norm"] != "none":
            x = x / ((x ** 2).mean(-1, keepdim=True) + 1e-6).sqrt()
        if s[n + "_weight"] is not None:
            x = x * s[n + "_weight"].double()
        if s[n + "_bias"] is not None:
            x = x + s[n + "_bias"].double()
        part = x[..., lo:hi]
        if c["interleaved"]:
            z = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous()) * turn
            part = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
            part = torch.cat([z.real, z.imag], -1)
        x[..., lo:hi] = part
        x[s["positions"] < 0] = 0.0  # left as they were
        out["out_" + n] = x
    return out


def _exact_store(c, s):
    bs, D, H = c["block"], c["dim"], c["heads"]
    values = _code_view(s["kv_cache"].view(torch.float8_e4m3fn), bs, D).double()  # [blocks, H, bs, 2, D]
    scales = _scale_view(s["kv_cache"], bs, D).double()
    x = torch.zeros_like(values)
    new = torch.zeros(values.shape[0], bs, dtype=torch.bool, device=DEV)
    at = torch.nonzero(s["slot_mapping"] >= 0).squeeze(-1)
    slot = s["slot_mapping"][at].long()
    blk, off = torch.div(slot, bs, rounding_mode="floor"), slot % bs
    new[blk, off] = True
    x[blk, :, off, 0], x[blk, :, off, 1] = s["k"][at].double(), s["v"][at].double()
    touched, fresh = new.any(-1)[:, None, None], new[:, 0][:, None, None]
    # the scale that the new tokens ask for is an f32 number by definition
    need = (x.abs().amax((2, 4)) / 448.0).float().double()
    up = torch.ceil(torch.log2(need.clamp(min=1e-300) / scales)).clamp(min=0)
    for d in (-1, 1):  # log2 next to a whole number: the first power at or above
        other = (up + d).clamp(min=0)
        up = torch.where((scales * 2.0 ** other >= need) & ((scales * 2.0 ** up < need) | (other < up)), other, up)
    up = torch.where(touched & ~fresh & (need > 0), up, torch.zeros_like(up))
    after = torch.where(fresh, need, scales * 2.0 ** up)
    before = (torch.arange(bs, device=DEV) < new.int().argmax(-1)[:, None]) & new.any(-1)[:, None]
    shifted = values * (0.5 ** up)[:, :, None, :, None]
    values = torch.where(before[:, None, :, None, None], shifted, values)
    values = torch.where(new[:, None, :, None, None], x / after.clamp(min=1e-300)[:, :, None, :, None], values)
    return {"codes": values, "scales": after}


def _exact_attn(c, s):
    bs, D, HK = c["block"], c["dim"], c["kv_heads"]
    G = c["heads"] // HK
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    cu, ctx = s["cu_new_lens"].tolist(), s["context_lens"].tolist()
    for b in range(c["requests"]):
        lo, hi, n = cu[b], cu[b + 1], ctx[b]
        pages = s["block_tables"][b, : -(-n // bs)].long()
        step = max(1, (1 << 28) // (n * G))
        for h in range(HK):
            page = s["kv_cache"][pages, h]
            e = page[:, : bs * 2 * D].reshape(-1, 2, D)[:n].view(torch.float8_e4m3fn).double()
            sc = page[:, bs * 2 * D: bs * 2 * D + 8].view(torch.float32).double().repeat_interleave(bs, 0)[:n]
            keys, vals = e[:, 0] * sc[:, :1], e[:, 1] * sc[:, 1:]
            for r in range(lo, hi, step):
                to = min(r + step, hi)
                w = torch.einsum("rgd,nd->rgn", s["q"][r:to, h * G: (h + 1) * G].double(), keys) * s["scale"]
                own_pos = torch.arange(r, to, device=DEV) - lo + n - (hi - lo)
                back = own_pos[:, None] - torch.arange(n, device=DEV)
                hidden = (back < 0) | (back >= (c["window"] or n + 1))
                w.masked_fill_(hidden[:, None], -math.inf)
                z = torch.logsumexp(w, -1)
                out[r:to, h * G: (h + 1) * G] = torch.einsum("rgn,nd->rgd", torch.exp_(w - z[..., None]), vals)
                lse[r:to, h * G: (h + 1) * G] = z
    return {"out": out, "lse": lse}


def exact(case, seed):
    """Outputs in 64 bits, written apart from the plain forms."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "store": _exact_store, "attn": _exact_attn}[case["op"]](case, s)
