"""Workloads of the operators around the FP8 indexer: a serving step's block
tables and slot maps, the quantising write into a paged cache, and the
attention over the selected positions of a paged cache.

Each case is one call of one operator on inputs as a serving loop has them.
With ``own`` false ``run`` computes the operator from elementary torch
operations; with ``own`` true it calls this package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a medium batch: every request adds one token
        {"name": "tables_decode_64", "op": "tables", "requests": 64, "new_max": 1, "rows": 64, "block": 64,
         "max_len": 32768},
        # a step that mixes prompt chunks and single tokens, small blocks
        {"name": "tables_chunk_8192", "op": "tables", "requests": 48, "new_max": 509, "rows": 8192, "block": 16,
         "max_len": 16384},
        # the largest step: as many requests as the calls accept, token slots
        {"name": "tables_4096_blk1", "op": "tables", "requests": 4096, "new_max": 63, "rows": 131072, "block": 1,
         "max_len": 2048},
        # index keys of a speculative decode step (16 requests of 6 rows)
        {"name": "store_index_96", "op": "store", "tokens": 96, "heads": 0, "dim": 128, "block": 64, "type": "bf16"},
        # index keys of a prompt chunk into the co-packed token cache
        {"name": "store_index_4096_blk1", "op": "store", "tokens": 4096, "heads": 0, "dim": 128, "block": 1,
         "type": "f32"},
        # keys and values of a large chunk, grouped heads
        {"name": "store_kv_16384", "op": "store", "tokens": 16384, "heads": 8, "dim": 128, "block": 64,
         "type": "bf16"},
        # one request, one token, short context: latency
        {"name": "attn_decode_1", "op": "attn", "form": "decode", "requests": 1, "next_n": 1, "heads": 32,
         "kv_heads": 1, "dim": 128, "block": 64, "length": 1024, "k": 512},
        # speculative verify: 16 requests of 6 rows over long contexts
        {"name": "attn_decode_mtp_verify", "op": "attn", "form": "decode", "requests": 16, "next_n": 6, "heads": 32,
         "kv_heads": 1, "dim": 128, "block": 64, "length": 131072, "k": 2048},
        # a large decode batch with grouped heads over the token cache
        {"name": "attn_decode_gqa_blk1", "op": "attn", "form": "decode", "requests": 64, "next_n": 4, "heads": 64,
         "kv_heads": 8, "dim": 128, "block": 1, "length": 32768, "k": 2048},
        # prompt chunks of four requests
        {"name": "attn_prefill_4x1024", "op": "attn", "form": "prefill", "requests": 4, "next_n": 1024, "heads": 32,
         "kv_heads": 1, "dim": 128, "block": 64, "length": 8192, "k": 2048},
        # odd sizes: short rows, three key heads, a k that fills no tile
        {"name": "attn_prefill_odd_d64", "op": "attn", "form": "prefill", "requests": 3, "next_n": 259, "heads": 21,
         "kv_heads": 3, "dim": 64, "block": 16, "length": 1531, "k": 500},
        # many query heads on one key head
        {"name": "attn_decode_h128", "op": "attn", "form": "decode", "requests": 32, "next_n": 2, "heads": 128,
         "kv_heads": 1, "dim": 128, "block": 32, "length": 16384, "k": 1024},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "store", "attn", "attn"])
    if op == "tables":
        requests = _log_int(rng, 1, 4096)
        new_max = _log_int(rng, 1, max(1, min(2048, 131072 // requests)))
        return {"op": op, "requests": requests, "new_max": new_max, "rows": requests * new_max + rng.randint(0, 300),
                "block": rng.choice([1, 16, 32, 64, 128]), "max_len": max(2 * new_max, _log_int(rng, 64, 8192))}
    if op == "store":
        heads = rng.choice([0, 1, 2, 3, 8])
        dim = rng.choice([64, 128])
        most = 16384 * 8 * 128 // (max(1, heads) * dim)
        return {"op": op, "tokens": _log_int(rng, 1, min(most, 32768)), "heads": heads, "dim": dim,
                "block": rng.choice([1, 16, 32, 64, 128]), "type": rng.choice(["bf16", "f16", "f32"])}
    form = rng.choice(["decode", "prefill"])
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 5, 7, 8, 16, 24, 32])
    k = _log_int(rng, 1, 2048)
    if form == "decode":
        requests, next_n = _log_int(rng, 1, 48), rng.randint(1, 6)
        length = _log_int(rng, max(16, next_n), 32768)
    else:
        requests, next_n = rng.randint(1, 4), _log_int(rng, 1, 512)
        length = next_n + _log_int(rng, 1, 4096)
    # no more scores than the largest listed case has
    group = max(1, min(group, 4096 * 2048 * 32 // (requests * next_n * k * kv_heads)))
    return {"op": op, "form": form, "requests": requests, "next_n": next_n, "heads": kv_heads * group,
            "kv_heads": kv_heads, "dim": rng.choice([64, 128]), "block": rng.choice([1, 16, 32, 64, 128]),
            "length": length, "k": k}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _quantise(x):
    """x [..., D] f32 -> e4m3 values (as float8) and f32 scales [...]."""
    amax = x.abs().amax(-1)
    scale = amax / E4M3_MAX
    codes = (x / scale.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(amax.unsqueeze(-1) == 0, torch.zeros_like(codes), codes)
    return codes.to(torch.float8_e4m3fn), scale


def page_bytes(block, dim, parts):
    """Bytes of a page of `block` tokens: the e4m3 rows of every token (keys,
    then values where the cache holds both), then the f32 scales; pages of a
    key/value cache are whole multiples of 16 bytes."""
    n = block * parts * (dim + 4)
    return n if parts == 1 else (n + 15) // 16 * 16


def _code_view(cache, block, dim, parts):
    """cache [..., page] u8 -> its e4m3 bytes [..., block, parts, dim]."""
    return cache[..., : block * parts * dim].unflatten(-1, (block, parts, dim))


def _scale_view(cache, block, dim, parts):
    """cache [..., page] u8 -> its scales [..., block, parts] f32."""
    at = block * parts * dim
    return cache[..., at: at + 4 * block * parts].view(torch.float32).unflatten(-1, (block, parts))


def _prepare_tables(c, seed):
    g = _gen(seed)
    B, bs = c["requests"], c["block"]
    max_blocks = -(-c["max_len"] // bs)
    new = torch.randint(1, c["new_max"] + 1, (B,), generator=g, device=DEV, dtype=torch.int64)
    new = torch.where(new.cumsum(0) <= c["rows"], new, torch.zeros_like(new))  # what does not fit waits
    old = (torch.rand(B, generator=g, device=DEV) * (c["max_len"] - c["new_max"] + 1)).long()
    has = (old + bs - 1) // bs
    need = (old + new + bs - 1) // bs
    total = int(need.sum())
    pool = torch.randperm(total + 64, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((B, max_blocks), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(max_blocks, device=DEV)[None, :] < has[:, None]
    n_held = int(has.sum())
    tables[held] = pool[:n_held]
    free = pool[n_held:].contiguous()
    s = {"old_lens": old.int(), "new_lens": new.int(), "free_blocks": free,
         "free_count": torch.tensor([free.numel()], dtype=torch.int32, device=DEV), "block_tables": tables,
         "context_lens": torch.empty(B, dtype=torch.int32, device=DEV),
         "cu_new_lens": torch.empty(B + 1, dtype=torch.int32, device=DEV),
         "slot_mapping": torch.empty(c["rows"], dtype=torch.int32, device=DEV),
         "counts": torch.empty(4, dtype=torch.int32, device=DEV),
         "cu_seq_lens": torch.empty(B + 1, dtype=torch.int32, device=DEV),
         "cu_seqlen_ks": torch.empty(c["rows"], dtype=torch.int32, device=DEV),
         "cu_seqlen_ke": torch.empty(c["rows"], dtype=torch.int32, device=DEV)}
    return s


_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _prepare_store(c, seed):
    g = _gen(seed)
    T, H, D, bs = c["tokens"], c["heads"], c["dim"], c["block"]
    parts = 1 if H == 0 else 2
    blocks = -(-T // bs) + 8
    shape = (T, D) if H == 0 else (T, H, D)
    x = [(torch.randn(shape, generator=g, device=DEV)
          * torch.exp(torch.randn(shape[:-1] + (1,), generator=g, device=DEV))).to(_TYPES[c["type"]])
         for _ in range(parts)]
    slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:T].int()
    slots = torch.where(torch.rand(T, generator=g, device=DEV) < 0.02, torch.full_like(slots, -1), slots)
    page = page_bytes(bs, D, parts)
    cache = torch.zeros((blocks, page) if H == 0 else (blocks, H, page), dtype=torch.uint8, device=DEV)
    return {"k": x[0], "v": x[1] if parts == 2 else None, "slot_mapping": slots, "kv_cache": cache}


def _fill_cache(cache, g, block, dim):
    """Keys and values ~ N(0, 1), one scale a row."""
    codes, scales = _code_view(cache, block, dim, 2), _scale_view(cache, block, dim, 2)
    rows = max(1, (1 << 28) // (codes[0].numel()))
    for at in range(0, cache.shape[0], rows):  # in parts: the f32 draws of a whole cache need not fit
        q, s = _quantise(torch.randn(codes[at: at + rows].shape, generator=g, device=DEV))
        codes[at: at + rows] = q.view(torch.uint8)
        scales[at: at + rows] = s


def _prepare_attn(c, seed):
    g = _gen(seed)
    B, n, H, HK, D, bs, k = (c[x] for x in ("requests", "next_n", "heads", "kv_heads", "dim", "block", "k"))
    L = c["length"]
    lens = (L - (torch.rand(B, generator=g, device=DEV) * 0.3 * (L - n)).long()) if c["form"] == "decode" else \
        torch.full((B,), L, dtype=torch.int64, device=DEV)
    max_blocks = -(-L // bs)
    blocks = B * max_blocks + 8
    cache = torch.zeros((blocks, HK, page_bytes(bs, D, 2)), dtype=torch.uint8, device=DEV)
    _fill_cache(cache, g, bs, D)
    tables = torch.randperm(blocks, generator=g, device=DEV)[: B * max_blocks].int().view(B, max_blocks)
    q = torch.randn((B, n, H, D), generator=g, device=DEV).to(torch.bfloat16)
    # the selection: neighbouring rows of a request agree on most positions
    pos = torch.arange(L, device=DEV)
    idx = torch.full((B, n, k), -1, dtype=torch.int32, device=DEV)
    m = min(k, L)
    for b in range(B):
        score = torch.randn(1, L, generator=g, device=DEV) + 0.3 * torch.randn(n, L, generator=g, device=DEV)
        last = lens[b] - n + torch.arange(n, device=DEV)  # the row's own position
        score = score.masked_fill(pos[None, :] > last[:, None], -math.inf)
        top = score.topk(m, dim=-1)
        sel = torch.where(top.values == -math.inf, torch.full_like(top.indices, L), top.indices).sort(-1).values
        idx[b, :, :m] = torch.where(sel == L, torch.full_like(sel, -1), sel).int()
    s = {"kv_cache": cache, "block_tables": tables, "scale": 1.0 / math.sqrt(D), "form": c["form"],
         "block": bs, "lse": torch.empty((B * n, H), dtype=torch.float32, device=DEV)}
    if c["form"] == "decode":
        s["q"], s["indices"] = q, idx.view(B * n, k)
        s["request"] = torch.arange(B, device=DEV).repeat_interleave(n)
    else:
        base = (torch.arange(B, device=DEV) * L).int()
        s["q"] = q.view(B * n, H, D)
        s["indices"] = torch.where(idx < 0, idx, idx + base[:, None, None]).view(B * n, k)
        s["cu_seq_lens"] = torch.cat([base, torch.tensor([B * L], dtype=torch.int32, device=DEV)])
    s["out"] = torch.empty_like(s["q"])
    return s


def prepare(case, seed):
    return {"op": case["op"], "case": dict(case),
            **{"tables": _prepare_tables, "store": _prepare_store, "attn": _prepare_attn}[case["op"]](case, seed)}


# -------------------------------------------------------------- plain forms
def _plain_tables(s):
    bs = s["case"]["block"]
    old, new = s["old_lens"].long(), s["new_lens"].long()
    tables, free, count = s["block_tables"], s["free_blocks"], s["free_count"].long()
    B, max_blocks = tables.shape
    rows = s["slot_mapping"].shape[0]
    dev = tables.device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    ctx = torch.minimum(old + new, torch.full_like(old, max_blocks * bs))
    has, need = (old + bs - 1) // bs, (ctx + bs - 1) // bs
    fresh = (need - has).clamp(min=0)
    first = fresh.cumsum(0) - fresh
    j = torch.arange(max_blocks, device=dev)[None, :]
    nth = first[:, None] + j - has[:, None]
    take = (j >= has[:, None]) & (j < need[:, None])
    got = torch.where(nth < count, free[(count - 1 - nth).clamp(0, free.shape[0] - 1)],
                      torch.full((1,), -1, dtype=torch.int32, device=dev))
    tables.copy_(torch.where(take, got, tables))
    cu_new = torch.cat([zero, new.cumsum(0)])
    cu_seq = torch.cat([zero, ctx.cumsum(0)])
    t = torch.arange(rows, device=dev)
    b = (torch.searchsorted(cu_new, t, right=True) - 1).clamp(0, B - 1)
    real = t < cu_new[B]
    pos = old[b] + t - cu_new[b]
    block = tables[b, (pos // bs).clamp(0, max_blocks - 1)].long()
    slot = torch.where(real & (pos < max_blocks * bs) & (block >= 0), block * bs + pos % bs, torch.full_like(t, -1))
    ks = torch.where(real, cu_seq[b], torch.zeros_like(t))
    ke = torch.where(real, cu_seq[b] + torch.minimum(pos + 1, ctx[b]), torch.zeros_like(t))
    taken = fresh.sum().reshape(1)
    missing = (taken - count).clamp(min=0)
    counts = torch.cat([cu_new[B:], taken - missing, count - (taken - missing), missing])
    return {"block_tables": tables, "context_lens": ctx.int(), "cu_new_lens": cu_new.int(),
            "slot_mapping": slot.int(), "counts": counts.int(), "cu_seq_lens": cu_seq.int(),
            "cu_seqlen_ks": ks.int(), "cu_seqlen_ke": ke.int()}


def _stored(s):
    """The cache's content as the values it stands for."""
    c = s["case"]
    parts = 1 if c["heads"] == 0 else 2
    return {"codes": _code_view(s["kv_cache"].view(torch.float8_e4m3fn), c["block"], c["dim"], parts),
            "scales": _scale_view(s["kv_cache"], c["block"], c["dim"], parts)}


def _plain_store(s):
    c = s["case"]
    bs, D = c["block"], c["dim"]
    parts = 1 if c["heads"] == 0 else 2
    slot = s["slot_mapping"].long()
    keep = slot >= 0
    blk, off = slot[keep] // bs, slot[keep] % bs
    codes, scales = _code_view(s["kv_cache"], bs, D, parts), _scale_view(s["kv_cache"], bs, D, parts)
    x = s["k"].unsqueeze(-2) if parts == 1 else torch.stack([s["k"], s["v"]], -2)
    q, sc = _quantise(x[keep].float())
    if parts == 1:
        codes[blk, off], scales[blk, off] = q.view(torch.uint8), sc
    else:
        codes[blk, :, off], scales[blk, :, off] = q.view(torch.uint8), sc
    return _stored(s)


def _attend(s, dtype):
    """Attention of every row over its selected positions, in `dtype`."""
    c = s["case"]
    bs, D, HK = c["block"], c["dim"], c["kv_heads"]
    idx, tables = s["indices"].long(), s["block_tables"].long()
    R, k = idx.shape
    q = s["q"].reshape(R, HK, -1, D).to(dtype)
    if c["form"] == "decode":
        req, tok = s["request"][:, None].expand(R, k), idx
    else:
        req = (torch.searchsorted(s["cu_seq_lens"].long(), idx, right=True) - 1).clamp(0, tables.shape[0] - 1)
        tok = idx - s["cu_seq_lens"].long()[req]
    ok = idx >= 0
    tok = tok.clamp(min=0)
    blk, off = tables[req, tok // bs], tok % bs
    codes = _code_view(s["kv_cache"], bs, D, 2)[blk, :, off].view(torch.float8_e4m3fn).to(dtype)  # [R, k, HK, 2, D]
    kv = codes * _scale_view(s["kv_cache"], bs, D, 2)[blk, :, off].to(dtype).unsqueeze(-1)
    score = torch.matmul(q, kv[:, :, :, 0].permute(0, 2, 3, 1)) * s["scale"]  # [R, HK, G, k]
    score = score.masked_fill(~ok[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[:, :, :, 1].permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    return out.reshape(s["q"].shape), (top + torch.log(total)).reshape(R, -1)


def _plain_attn(s):
    out, lse = _attend(s, torch.float32)
    return {"out": out.to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------------------- runs
def run(state):
    s = state
    if own:
        import sparse_attention_fp8_gb300 as fp8idx
        if s["op"] == "tables":
            fp8idx.paged_step_tables(s["old_lens"], s["new_lens"], s["free_blocks"], s["free_count"],
                                     s["case"]["block"], s["block_tables"], s["context_lens"], s["cu_new_lens"],
                                     s["slot_mapping"], s["counts"], cu_seq_lens=s["cu_seq_lens"],
                                     cu_seqlen_ks=s["cu_seqlen_ks"], cu_seqlen_ke=s["cu_seqlen_ke"])
            return {n: s[n] for n in ("block_tables", "context_lens", "cu_new_lens", "slot_mapping", "counts",
                                      "cu_seq_lens", "cu_seqlen_ks", "cu_seqlen_ke")}
        if s["op"] == "store":
            fp8idx.fp8_paged_store(s["k"], s["v"], s["slot_mapping"], s["kv_cache"])
            return _stored(s)
        if s["form"] == "decode":
            fp8idx.fp8_paged_sparse_attn(s["q"], s["kv_cache"], s["indices"], s["block_tables"], s["scale"],
                                         s["out"], lse=s["lse"])
        else:
            fp8idx.fp8_mqa_sparse_attn_paged(s["q"], s["kv_cache"], s["block_tables"], s["cu_seq_lens"],
                                             s["indices"], s["scale"], s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"tables": _plain_tables, "store": _plain_store, "attn": _plain_attn}[s["op"]](s)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "tables":
        B, T, bs = c["requests"], c["rows"], c["block"]
        new_tokens = min(T, B * (c["new_max"] + 1) // 2)
        fresh = new_tokens // bs + B // 2
        # lengths, the free blocks dealt and their table entries, a table
        # entry per block that holds new tokens, and the outputs
        return {"bytes": 8 * B + 8 * fresh + 4 * (new_tokens // bs + B) + 12 * B + 12 * T + 24, "flops": 0}
    if c["op"] == "store":
        rows = c["tokens"] * max(1, c["heads"]) * (1 if c["heads"] == 0 else 2)
        size = 4 if c["type"] == "f32" else 2
        return {"bytes": rows * (c["dim"] * size + c["dim"] + 4) + 4 * c["tokens"], "flops": 2 * rows * c["dim"]}
    R = c["requests"] * c["next_n"]
    picked = min(c["k"], c["length"])
    # a request's rows together read at least one row's selection; a chunk's
    # rows pick every position of the window between them
    union = picked if c["form"] == "decode" else min(c["length"], R * picked)
    kv = c["requests"] * union * c["kv_heads"] * (2 * c["dim"] + 8)
    io = R * (2 * c["heads"] * c["dim"] * 2 + 4 * c["heads"] + 4 * c["k"])
    return {"bytes": kv + io, "flops": 4 * R * c["heads"] * picked * c["dim"]}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """Outputs in 64 bits, written apart from the plain forms."""
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    c = case
    bs, D = c["block"], c["dim"]
    if c["op"] == "store":
        parts = 1 if c["heads"] == 0 else 2
        blocks = s["kv_cache"].shape[0]
        shape = (blocks, bs, parts, D) if parts == 1 else (blocks, c["heads"], bs, parts, D)
        codes = torch.zeros(shape, dtype=torch.float64, device=DEV)
        scales = torch.zeros(shape[:-1], dtype=torch.float64, device=DEV)
        at = torch.nonzero(s["slot_mapping"] >= 0).squeeze(-1)
        blk = torch.div(s["slot_mapping"][at].long(), bs, rounding_mode="floor")
        off = s["slot_mapping"][at].long() - blk * bs
        for part, x in enumerate((s["k"], s["v"])[:parts]):
            x = x[at].double()
            sc = x.abs().max(dim=-1).values / 448.0
            value = x / sc.clamp(min=1e-300)[..., None]  # the value a code stands for, before its rounding
            if parts == 1:
                codes[blk, off, 0], scales[blk, off, 0] = value, sc
            else:
                codes[blk, :, off, part], scales[blk, :, off, part] = value, sc
        return {"codes": codes, "scales": scales}
    R, k = s["indices"].shape
    HK, G = c["kv_heads"], c["heads"] // c["kv_heads"]
    out = torch.zeros(R, c["heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((R, c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    per_request = R // c["requests"]
    step = max(1, (1 << 30) // (k * HK * 2 * D * 8 + 8 * k * c["heads"]))
    code_bytes = s["kv_cache"][..., : bs * 2 * D]
    scale_bytes = s["kv_cache"][..., bs * 2 * D: bs * 2 * D + 8 * bs].view(torch.float32)
    for b in range(c["requests"]):
        base = b * c["length"] if c["form"] == "prefill" else 0
        row_of = s["block_tables"][b].long()
        for lo in range(b * per_request, (b + 1) * per_request, step):
            hi = min(lo + step, (b + 1) * per_request)
            idx = s["indices"][lo:hi].long()
            ok = idx >= 0
            tok = torch.where(ok, idx - base, torch.zeros_like(idx))
            page, t = row_of[torch.div(tok, bs, rounding_mode="floor")], tok % bs
            at = t[..., None] * (2 * D) + torch.arange(2 * D, device=DEV)
            for h in range(HK):
                e = code_bytes[:, h][page[..., None], at].view(torch.float8_e4m3fn).double()
                keys = e[..., :D] * scale_bytes[:, h][page, 2 * t].double()[..., None]
                vals = e[..., D:] * scale_bytes[:, h][page, 2 * t + 1].double()[..., None]
                qh = s["q"].reshape(R, c["heads"], D)[lo:hi, h * G: (h + 1) * G].double()
                w = torch.einsum("rgd,rkd->rgk", qh, keys) * s["scale"]
                w = torch.where(ok[:, None, :], w, torch.full_like(w, -math.inf))
                z = torch.logsumexp(w, -1)
                p = torch.where(ok[:, None, :], torch.exp(w - z[..., None]), torch.zeros_like(w))
                out[lo:hi, h * G: (h + 1) * G] = torch.einsum("rgk,rkd->rgd", p, vals)
                lse[lo:hi, h * G: (h + 1) * G] = z
    return {"out": out.reshape(s["q"].shape), "lse": lse}
