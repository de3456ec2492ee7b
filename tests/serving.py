"""Cases and tolerances for the tests of the operators around the indexer.

The attention's error bound, per output, from what the kernel rounds:
  * the output's own rounding to bf16: 2^-8 of the value (half a step);
  * a probability is held as two e4m3 values of 4 significant bits each, so
    it is off by at most 2^-8 of itself, and by at most 2^-19 of the largest
    probability (times the largest value scale) where it is so small that
    the e4m3 range ends;
  * a score of D <= 128 products summed in f32 is off by at most 2^-16 of the
    sum of its |products| (128 f32 additions of 2^-24 each for either part, a
    few more to join and scale them; the query's two e4m3 parts are exact,
    but for elements below 2^-10 of their head's largest one, which are off by
    at most 2^-18 of that and of which a row of 64 or 128 normal values has
    one at most), which changes a probability by the same relative amount;
    2^-20 covers the exponential and the f32 sums;
so |error| <= 2^-8 |out| + (2^-8 + 2^-20 + 2 * 2^-16 S) sum w|v|
              + 2^-19 * floor, all but the first times (1 + 2^-7) for the
second order, with S the largest sum of |products| of a score.
The log-sum-exp is off by 2^-16 (1 + S) at most.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import serving as ref


def bf16(x):
    """f32 array rounded to bf16 values (kept as f32)."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def filled_cache(rng, blocks, kv_heads, block_size, dim, spread=0.3):
    """A key/value cache with every slot written: N(0, 1) rows times
    exp(spread * N(0, 1))."""
    cache = rng.integers(0, 256, (blocks, kv_heads, ref.page_bytes(block_size, dim)), dtype=np.uint8)
    n = blocks * block_size
    k = rng.standard_normal((n, kv_heads, dim)) * np.exp(spread * rng.standard_normal((n, kv_heads, 1)))
    v = rng.standard_normal((n, kv_heads, dim)) * np.exp(spread * rng.standard_normal((n, kv_heads, 1)))
    for part, x in enumerate((k, v)):
        codes, scale = ref.quantise_rows(x)
        codes = codes.reshape(blocks, block_size, kv_heads, dim).transpose(0, 2, 1, 3)
        scale = scale.reshape(blocks, block_size, kv_heads).transpose(0, 2, 1)
        cache[..., : block_size * 2 * dim].reshape(blocks, kv_heads, block_size, 2, dim)[:, :, :, part] = codes
        at = block_size * 2 * dim
        sc = np.ascontiguousarray(cache[..., at: at + 8 * block_size]).view(np.float32)
        sc = sc.reshape(blocks, kv_heads, block_size, 2)
        sc[..., part] = scale
        cache[..., at: at + 8 * block_size] = sc.reshape(blocks, kv_heads, -1).view(np.uint8)
    return cache


def assert_attention(out, lse, want, what=""):
    """out [R, H, D] f32 (bf16 values) and lse [R, H] against
    ref.sparse_attention's figures."""
    o, z, mag, floor, sabs = want
    assert np.isfinite(out).all(), f"{what}: non-finite outputs"
    S = sabs[..., None]
    tol = 2.0**-8 * np.abs(o) + (1 + 2.0**-7) * ((2.0**-8 + 2.0**-20 + 2 * 2.0**-16 * S) * mag + 2.0**-19 * floor)
    err = np.abs(out.astype(np.float64) - o)
    bad = err > tol + 1e-30
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outputs off; worst {float((err - tol).max()):.3g} "
                           f"over, at {np.unravel_index(np.argmax(err - tol), err.shape)}")
    none = np.isneginf(z)
    assert np.array_equal(np.isneginf(lse), none), f"{what}: rows without entries"
    assert (out[none] == 0).all(), f"{what}: a row without entries is not 0"
    e = np.abs(lse[~none].astype(np.float64) - z[~none])
    assert (e <= 2.0**-16 * (1 + sabs[~none])).all(), f"{what}: lse off by {float(e.max()):.3g}"
