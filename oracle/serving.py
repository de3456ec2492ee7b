"""Plain CPU definitions of the operators around the indexer: step tables,
the quantising paged store and the attention over selected positions
(numpy, 64 bits, loops where they are clearest).  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np
import torch

INT_MAX = 2**31 - 1


def step_tables(old_lens, new_lens, free_blocks, free_count, block_size, block_tables, rows):
    """Every output of a step as a dict; block_tables is not changed."""
    tables = block_tables.copy()
    B, max_blocks = tables.shape
    cap = max_blocks * block_size
    count = int(min(max(int(free_count), 0), len(free_blocks)))
    ctx, cu_new, cu_seq = [], [0], [0]
    wanted = 0
    slots, ks, ke = [], [], []
    for b in range(B):
        old, new = max(int(old_lens[b]), 0), max(int(new_lens[b]), 0)
        c = min(old + new, cap)
        for j in range(-(-old // block_size), -(-c // block_size)):
            tables[b, j] = free_blocks[count - 1 - wanted] if wanted < count else -1
            wanted += 1
        for i in range(min(new, rows - len(slots))):  # (rows past the outputs are dropped)
            pos = old + i
            slot = -1
            if pos < cap and tables[b, pos // block_size] >= 0:
                slot = int(tables[b, pos // block_size]) * block_size + pos % block_size
            slots.append(slot if slot <= INT_MAX else -1)
            ks.append(min(cu_seq[-1], INT_MAX))
            ke.append(min(cu_seq[-1] + min(pos + 1, c), INT_MAX))
        ctx.append(c)
        cu_new.append(cu_new[-1] + new)
        cu_seq.append(cu_seq[-1] + c)
    pad = rows - len(slots)
    dealt = min(wanted, count)
    arr = lambda v: np.minimum(np.asarray(v, np.int64), INT_MAX).astype(np.int32)  # noqa: E731
    return {"block_tables": tables, "context_lens": arr(ctx), "cu_new_lens": arr(cu_new), "cu_seq_lens": arr(cu_seq),
            "slot_mapping": arr(slots + [-1] * pad), "cu_seqlen_ks": arr(ks + [0] * pad),
            "cu_seqlen_ke": arr(ke + [0] * pad),
            "counts": arr([cu_new[-1], dealt, count - dealt, wanted - dealt])}


def quantise_rows(x):
    """x [..., D] f32 -> (e4m3 codes u8 [..., D], scales f32 [...]): scale =
    max|x| / 448 (NaN do not count) and x / scale in f32, codes rounded to
    nearest even, NaN codes for NaN."""
    x = np.asarray(x, np.float32)
    amax = np.fmax.reduce(np.abs(x), axis=-1, initial=0)
    scale = (amax / np.float32(448)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where((amax[..., None] == 0) & ~np.isnan(x), np.float32(0), x / scale[..., None]).astype(np.float32)
    y = np.clip(y, -448, 448)
    return torch.from_numpy(np.ascontiguousarray(y)).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale


def e4m3_values():
    """The value of each of the 256 codes (NaN for S.1111.111)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e == 15 and m == 7) else (m / 8.0 * 2.0**-6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        out[c] = -v if c >> 7 else v
    return out


def page_bytes(block_size, dim):
    return -(-block_size * (2 * dim + 8) // 16) * 16


def store_kv(cache, slots, k, v, block_size):
    """cache [num_blocks, kv_heads, page] u8, changed in place; k, v [T, kv_heads, D]."""
    D = k.shape[-1]
    for part, x in enumerate((k, v)):
        codes, scale = quantise_rows(x)
        for t, s in enumerate(slots):
            if not 0 <= s < cache.shape[0] * block_size:
                continue
            b, o = divmod(int(s), block_size)
            for h in range(cache.shape[1]):
                at = (2 * o + part) * D
                cache[b, h, at: at + D] = codes[t, h]
                at = block_size * 2 * D + 4 * (2 * o + part)
                cache[b, h, at: at + 4] = scale[t, h: h + 1].view(np.uint8)


def store_index(cache, slots, k, block_size):
    """cache [num_blocks, block_size*(D+4)] u8, changed in place; k [T, D]."""
    D = k.shape[-1]
    codes, scale = quantise_rows(k)
    for t, s in enumerate(slots):
        if not 0 <= s < cache.shape[0] * block_size:
            continue
        b, o = divmod(int(s), block_size)
        cache[b, o * D: (o + 1) * D] = codes[t]
        at = block_size * D + 4 * o
        cache[b, at: at + 4] = scale[t: t + 1].view(np.uint8)


def selected(idx, row, block_tables, block_size, num_blocks, next_n=None, cu_seq_lens=None):
    """(block, offset) of every selected entry of one row's indices."""
    out = []
    for i in idx.tolist():
        if i < 0:
            continue
        if cu_seq_lens is None:
            req, tok = row // next_n, i
        else:
            req = int(np.searchsorted(cu_seq_lens, i, side="right")) - 1
            if req < 0 or req >= len(cu_seq_lens) - 1:
                continue
            tok = i - int(cu_seq_lens[req])
        if tok // block_size >= block_tables.shape[1]:
            continue
        b = int(block_tables[req, tok // block_size])
        if 0 <= b < num_blocks:
            out.append((b, tok % block_size))
    return out


def sparse_attention(q, cache, indices, block_tables, block_size, scale, next_n=None, cu_seq_lens=None, by_product=False):
    """q [R, H, D] f64, cache [num_blocks, kv_heads, page] u8.  Returns out
    [R, H, D], lse [R, H] and three figures that an error bound needs: the
    sum of weight * |value| per output [R, H, D], the largest weight times
    the largest value scale (by_product: the largest product of an entry's
    weight and value scale) times the sum of |value code| [R, H, D], and the
    largest sum of |scale * q * k| of a score [R, H]."""
    R, H, D = q.shape
    HK = cache.shape[1]
    G = H // HK
    table = e4m3_values()
    out, lse = np.zeros((R, H, D)), np.full((R, H), -np.inf)
    mag, floor, sabs = np.zeros((R, H, D)), np.zeros((R, H, D)), np.zeros((R, H))
    for r in range(R):
        sel = selected(indices[r], r, block_tables, block_size, cache.shape[0], next_n, cu_seq_lens)
        if not sel:
            continue
        for g in range(HK):
            rows = np.stack([cache[b, g, o * 2 * D: (o + 1) * 2 * D] for b, o in sel])
            at = block_size * 2 * D
            sc = np.stack([cache[b, g, at + 8 * o: at + 8 * o + 8].copy().view(np.float32) for b, o in sel]).astype(
                np.float64)
            codes = table[rows]
            key = codes[:, :D] * sc[:, :1]
            val = codes[:, D:] * sc[:, 1:]
            for h in range(g * G, (g + 1) * G):
                s = scale * (key @ q[r, h])
                top = s.max()
                z = np.exp(s - top).sum()
                w = np.exp(s - top) / z
                lse[r, h] = top + np.log(z)
                out[r, h] = w @ val
                mag[r, h] = w @ np.abs(val)
                most = (w * np.abs(sc[:, 1])).max() if by_product else w.max() * np.abs(sc[:, 1]).max()
                floor[r, h] = most * np.abs(codes[:, D:]).sum(0)
                sabs[r, h] = (np.abs(scale) * (np.abs(key) @ np.abs(q[r, h]))).max()
    return out, lse, mag, floor, sabs
