"""Cases and tolerances for the tests of the block-scaled cache's operators.

The attention's error bound, per output, from what the kernel rounds (S: the
largest sum of |products| of a score, `mag` the sum of weight * |value|,
`floor` the largest product of a weight and a value scale times the sum of the
|value codes|):
  * the output's own rounding to bf16: 2^-8 of the value (half a step);
  * a probability times its value's scale is held as f16: off by at most 2^-11
    of itself, and where it is subnormal by half a step of 2^-24, 2^-25 of a
    reference that is less than twice the row's largest one: 2^-24 floor;
  * a score of D <= 128 products summed in f32 is off by at most 2^-16 of the
    sum of its |products| (the query's two e4m3 parts are exact, but for
    elements below 2^-10 of their head's largest one, off by at most 2^-17 of
    that, and of which a row of 64 or 128 normal values has one at most), which
    changes a probability by the same relative amount; so do the roundings of
    the exponent (f32 numbers of the size of the scores: 2^-22 S);
  * 2^-16 covers the logarithms of the value scales (numbers up to 64 in f32),
    the exponential and the f32 sums;
so |error| <= 2^-8 |out| + (1 + 2^-7) ((2^-11 + 2^-16 + 2 * 2^-16 S) mag
              + 2^-24 floor), the factor for the second order.
The log-sum-exp is off by 2^-16 (1 + S) at most.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import serving as ref


def filled_blocks(rng, blocks, kv_heads, block_size, dim, spread=0.3):
    """A cache with every slot written and the bytes without meaning random:
    N(0, 1) rows times exp(spread * N(0, 1))."""
    cache = rng.integers(0, 256, (blocks, kv_heads, ref.block_page_bytes(block_size, dim)), dtype=np.uint8)
    x = rng.standard_normal((blocks, kv_heads, block_size, 2, dim)).astype(np.float32)
    x *= np.exp(spread * rng.standard_normal((blocks, kv_heads, block_size, 2, 1))).astype(np.float32)
    scale = (np.abs(x).max((2, 4)) / np.float32(448)).astype(np.float32)
    codes = torch.from_numpy(np.clip(x / scale[:, :, None, :, None], -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    at = block_size * 2 * dim
    cache[..., :at] = codes.numpy().reshape(blocks, kv_heads, -1)
    cache[..., at: at + 8] = scale.view(np.uint8).reshape(blocks, kv_heads, 8)
    return cache


def scales_of(cache, block_size, dim):
    """The [blocks, kv_heads, 2] f32 scales of a cache (a copy)."""
    at = block_size * 2 * dim
    return np.ascontiguousarray(cache[..., at: at + 8]).view(np.float32)


def set_scales(cache, block_size, dim, scales):
    at = block_size * 2 * dim
    cache[..., at: at + 8] = np.ascontiguousarray(scales, np.float32).view(np.uint8)


def assert_block_attention(out, lse, want, what=""):
    """out [R, H, D] f32 (bf16 values) and lse [R, H] against
    ref.block_attention's figures; rows that are no request's must be NaN, as
    they were before the call."""
    o, z, mag, floor, sabs = want
    past = np.isnan(z).all(1)
    assert np.isnan(out[past]).all() and np.isnan(lse[past]).all(), f"{what}: rows past the requests were written"
    o, z, mag, floor, sabs, out, lse = (x[~past] for x in (o, z, mag, floor, sabs, out, lse))
    assert np.isfinite(out).all(), f"{what}: non-finite outputs"
    S = sabs[..., None]
    tol = 2.0**-8 * np.abs(o) + (1 + 2.0**-7) * ((2.0**-11 + 2.0**-16 + 2 * 2.0**-16 * S) * mag + 2.0**-24 * floor)
    err = np.abs(out.astype(np.float64) - o)
    bad = err > tol + 1e-30
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outputs off; worst {float((err - tol).max()):.3g} "
                           f"over, at {np.unravel_index(np.argmax(err - tol), err.shape)}")
    none = np.isneginf(z)
    assert np.array_equal(np.isneginf(lse), none), f"{what}: rows without positions"
    assert (out[none] == 0).all(), f"{what}: a row without positions is not 0"
    e = np.abs(lse[~none].astype(np.float64) - z[~none])
    assert (e <= 2.0**-16 * (1 + sabs[~none])).all(), f"{what}: lse off by {float(e.max()):.3g}"
