"""The attention over selected positions where values, weights or queries of
one row lie far apart, against 64-bit numpy.  The bound is that of serving.py
with the last step of the codes counted against the largest product of an
entry's probability and value scale (not against the largest of each): that
product has a code of 32 or more where the last step is 2^-13, half of which
is 2^-19 of it."""
import numpy as np
import pytest
import torch

from oracle import serving as ref
from serving import assert_attention, bf16
from test_sparse_attn_gpu import pick, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    m.device_status()
    return m


def attend(fp8idx, q, cache, idx, tables, bs, scale, ctas=0, what=""):
    """q [B, n, H, D] f32, rounded to bf16 for both sides."""
    q = bf16(q)
    B, n, H, D = q.shape
    out = torch.full((B, n, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B * n, H), float("nan"), device="cuda")
    fp8idx.fp8_paged_sparse_attn(torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(),
                                 torch.from_numpy(idx).cuda(), torch.from_numpy(tables).cuda(), scale, out, lse=lse,
                                 options=fp8idx.Options(num_ctas=ctas) if ctas else None)
    torch.cuda.synchronize()
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
    want = ref.sparse_attention(q.reshape(B * n, H, D).astype(np.float64), cache, idx, tables, bs, scale, next_n=n,
                                by_product=True)
    assert_attention(out.float().cpu().numpy().reshape(B * n, H, D), lse.cpu().numpy(), want, what)


def scales_of(cache, bs, D):
    """The cache's scales [num_blocks, kv_heads, bs, 2] (a copy), and a
    function that writes them back."""
    at = bs * 2 * D
    sc = np.ascontiguousarray(cache[..., at: at + 8 * bs]).view(np.float32).reshape(*cache.shape[:2], bs, 2)

    def put():
        cache[..., at: at + 8 * bs] = np.ascontiguousarray(sc).reshape(*cache.shape[:2], -1).view(np.uint8)
    return sc, put


def at(tables, pos, bs, req=0):
    return int(tables[req, pos // bs]), pos % bs


def aligned_keys(cache, tables, bs, D, score, length):
    """Makes every key of request 0 a multiple of the all-ones row, so that a
    query of ones over D scores score[i] at position i."""
    sc, put = scales_of(cache, bs, D)
    code = ref.quantise_rows(np.ones((1, D)))[0][0]   # 448 each
    for i in range(length):
        b, o = at(tables, i, bs)
        cache[b, :, o * 2 * D: o * 2 * D + D] = code
        sc[b, :, o, 0] = np.float32(score[i]) / 448
    put()


@pytest.mark.parametrize("H", [3, 20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [-75, -60, -40, -20, -12, -8, -3, 3, 8, 12, 20, 40, 60, 75])
@pytest.mark.parametrize("score", [20.0, 30.0])
def test_two_entries_of_far_apart_values(fp8idx, D, H, bits, score):
    """Scores that differ by 40 or 60, values that differ by 2^bits: whichever
    product of weight and value is larger keeps its bits."""
    rng = np.random.default_rng(bits + 100)
    q, cache, tables = setup(rng, 1, 1, H, 1, D, 16, 16, extra=0)
    q[:] = 1.0 / D
    aligned_keys(cache, tables, 16, D, [score, -score] + [0.0] * 14, 16)
    sc, put = scales_of(cache, 16, D)
    sc[..., 1] = 1.0 / 448
    sc[tables[0, 0], 0, 1, 1] *= np.float32(2.0**bits)
    put()
    for ctas in (0, 1, 2):
        attend(fp8idx, q, cache, np.array([[0, 1]], np.int32), tables, 16, 1.0, ctas=ctas, what=f"{ctas} CTAs")


def spread_rows(fp8idx, rng, rows, H, D, length, score, gain, bs=16):
    """`rows` rows of one request that all select 0 .. length-1, keys with the
    given scores, value scales times `gain`, as clusters and as persistent
    CTAs (many rows)."""
    q, cache, tables = setup(rng, 1, 1, H, 2, D, bs, length, extra=0, spread=0.2)
    q[:] = 1.0 / D
    q = np.repeat(q, rows, axis=1) * rng.uniform(0.9, 1.1, (1, rows, H, 1))
    aligned_keys(cache, tables, bs, D, score, length)
    sc, put = scales_of(cache, bs, D)
    for i in range(length):
        b, o = at(tables, i, bs)
        sc[b, :, o, 1] *= np.float32(gain[i])
    put()
    idx = np.tile(np.arange(length, dtype=np.int32), (rows, 1))
    for ctas in (0, 1, 4) if rows == 1 else (0,):
        attend(fp8idx, q, cache, idx, tables, bs, 1.0, ctas=ctas, what=f"{ctas} CTAs")


@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("where", [3, 300, 599])
@pytest.mark.parametrize("bits", [-30, -14, -5, 14])
def test_one_heavy_entry_of_another_size(fp8idx, where, bits, H):
    """One entry with nearly all the weight and values of another size, in
    the first, a middle and the last tile."""
    rng = np.random.default_rng(where + bits + 50)
    score, gain = rng.standard_normal(600), np.ones(600)
    score[where], gain[where] = 25.0, 2.0**bits
    spread_rows(fp8idx, rng, 1, H, 128, 600, score, gain)


@pytest.mark.parametrize("rows,length", [(1, 600), (330, 270)])
@pytest.mark.parametrize("gain0", [0.0, 2.0**-30, 2.0**-7])
@pytest.mark.parametrize("D", [64, 128])
def test_a_heavy_entry_of_little_value(fp8idx, D, gain0, rows, length):
    """Most of the weight on an entry whose values are zero or small: the
    output is made of the others."""
    rng = np.random.default_rng(7)
    score, gain = rng.standard_normal(length), np.ones(length)
    score[0], gain[0] = 18.0, gain0
    spread_rows(fp8idx, rng, rows, 4, D, length, score, gain)


@pytest.mark.parametrize("step", [-9, -3, 3, 9])
@pytest.mark.parametrize("slope", [-9.0, -2.0, 0.0, 2.0, 9.0])
def test_value_sizes_and_scores_that_change_from_tile_to_tile(fp8idx, step, slope):
    rng = np.random.default_rng(int(step * 10 + slope) + 200)
    tile = np.arange(900) // 128
    spread_rows(fp8idx, rng, 1, 20, 64, 900, rng.standard_normal(900) + slope * tile, 2.0**(step * tile))


@pytest.mark.parametrize("rows", [2, 330])
@pytest.mark.parametrize("D,H", [(128, 5), (64, 40)])
def test_any_value_sizes(fp8idx, rows, D, H):
    """Value rows of sizes e^(3 N(0, 1)), scales of either sign, some zero."""
    rng = np.random.default_rng(rows + D)
    q, cache, tables = setup(rng, 1, rows, H, 1, D, 16, 700, spread=0.3)
    sc, put = scales_of(cache, 16, D)
    sc[..., 1] *= np.exp(3 * rng.standard_normal(sc.shape[:-1])) * rng.choice([-1, 1, 0], sc.shape[:-1], p=[0.4, 0.55, 0.05])
    put()
    idx = pick(rng, rows, 400, 700)
    idx[rng.random(idx.shape) < 0.1] = -1
    for ctas in (0, 1, 2) if rows == 2 else (0,):
        attend(fp8idx, q, cache, idx, tables, 16, 1.5 * D**-0.5, ctas=ctas, what=f"{ctas} CTAs")


def test_rows_of_near_and_far_apart_values_in_turn(fp8idx):
    """Persistent CTAs: a row's reference does not reach the next row."""
    rng = np.random.default_rng(41)
    rows, D, bs = 700, 128, 16
    q, cache, tables = setup(rng, 1, rows, 6, 1, D, bs, 640, extra=0, spread=0.2)
    sc, put = scales_of(cache, bs, D)
    for i in range(320, 640):
        b, o = at(tables, i, bs)
        sc[b, :, o, 1] *= np.float32(2.0**int(rng.integers(-30, 31)))
    put()
    idx = np.sort(rng.integers(0, 320, (rows, 200)), axis=1).astype(np.int32)
    far = rng.random(rows) < 0.4
    idx[far] += 320
    attend(fp8idx, q, cache, idx, tables, bs, 0.09)


def test_all_values_zero(fp8idx):
    rng = np.random.default_rng(42)
    q, cache, tables = setup(rng, 1, 2, 4, 1, 64, 16, 300)
    sc, put = scales_of(cache, 16, 64)
    sc[..., 1] = 0
    put()
    for ctas in (0, 2):
        attend(fp8idx, q, cache, pick(rng, 2, 290, 300), tables, 16, 0.1, ctas=ctas)


@pytest.mark.parametrize("where", [0, 200, 599])
@pytest.mark.parametrize("score", [30.0, 50.0, 70.0, 150.0])
def test_entries_without_values_bound_no_sum(fp8idx, score, where):
    """Zero values with a score so far above the others' that the
    exponentials over a reference made of the others would overflow."""
    rng = np.random.default_rng(where + int(score))
    scores, gain = rng.standard_normal(600), np.ones(600)
    scores[where], gain[where] = score, 0.0
    scores[where - 1], gain[where - 1] = score - 1.0, 0.0
    spread_rows(fp8idx, rng, 1, 4, 128, 600, scores, gain)


@pytest.mark.parametrize("first", [0.0, 2.0**-70, 2.0**70])
def test_first_tile_of_other_values(fp8idx, first):
    """The reference of the value scales is the first tile's largest."""
    rng = np.random.default_rng(43)
    gain = np.where(np.arange(600) < 256, first, 1.0)
    for slope in (0.0, 48.0 if first > 1 else 0.0):
        spread_rows(fp8idx, rng, 1, 20, 128, 600, rng.standard_normal(600) + slope * (np.arange(600) >= 256), gain)


@pytest.mark.parametrize("ctas", [1, 2])
def test_partial_sums_over_far_apart_references(fp8idx, ctas):
    """Tiles without values on one of a row's pipelines; on the other, values
    that grow by 2^60 under falling scores: their references lie 2^130 apart,
    their weights do not."""
    rng = np.random.default_rng(46)
    tile = np.arange(1024) // 128
    score = np.where((tile == 3) | (tile == 7), -25.0, 0.0) + 0.1 * rng.standard_normal(1024)
    gain = np.array([0.0, 1.0, 0.0, 2.0**60, 0.0, 1.0, 0.0, 2.0**60])[tile]
    q, cache, tables = setup(rng, 1, 1, 6, 1, 128, 16, 1024, extra=0, spread=0.2)
    q[:] = 1.0 / 128
    aligned_keys(cache, tables, 16, 128, score, 1024)
    sc, put = scales_of(cache, 16, 128)
    for i in range(1024):
        b, o = at(tables, i, 16)
        sc[b, :, o, 1] *= np.float32(gain[i])
    put()
    attend(fp8idx, q, cache, np.arange(1024, dtype=np.int32)[None], tables, 16, 1.0, ctas=ctas)


def test_a_reference_that_rises_by_more_than_a_float_holds(fp8idx):
    """Little values of no weight, then weight without values, then values:
    the reference rises by 2^127 at once over sums that stay in range."""
    rng = np.random.default_rng(47)
    tile = np.arange(768) // 128
    score = np.array([-130.0, -130.0, 24.0, 24.0, 22.4, 22.4])[tile] + 0.1 * rng.standard_normal(768)
    spread_rows(fp8idx, rng, 1, 6, 128, 768, score, np.array([2.0**-17, 2.0**-17, 0.0, 0.0, 1.0, 1.0])[tile])


def test_a_scale_past_the_span_becomes_the_reference(fp8idx):
    """Values 2^100 times as large as all before, then of that size."""
    rng = np.random.default_rng(44)
    spread_rows(fp8idx, rng, 1, 6, 64, 700, rng.standard_normal(700), np.where(np.arange(700) < 300, 1.0, 2.0**100))
    spread_rows(fp8idx, rng, 1, 6, 64, 700, rng.standard_normal(700), np.where(np.arange(700) < 300, 0.0, 2.0**100))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctas", [0, 1, 4])
def test_value_scales_that_are_no_numbers(fp8idx, value, ctas):
    """They make the outputs of the rows that select them NaN; the scores'
    log-sum-exp does not depend on them."""
    rng = np.random.default_rng(45)
    q, cache, tables = setup(rng, 1, 2, 6, 1, 128, 16, 700, spread=0.3)
    idx = np.tile(np.arange(600, dtype=np.int32), (2, 1))
    idx[0, 333] = 650
    want = ref.sparse_attention(q.reshape(2, 6, 128).astype(np.float64), cache, idx, tables, 16, 0.3, next_n=2, by_product=True)
    sc, put = scales_of(cache, 16, 128)
    b, o = at(tables, 650, 16)
    sc[b, 0, o, 1] = value
    put()
    out = torch.empty((1, 2, 6, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 6), device="cuda")
    fp8idx.fp8_paged_sparse_attn(torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(),
                                 torch.from_numpy(idx).cuda(), torch.from_numpy(tables).cuda(), 0.3, out, lse=lse,
                                 options=fp8idx.Options(num_ctas=ctas))
    got, z = out[0].float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(got[0]).all()
    assert (np.abs(z[0] - want[1][0]) <= 2.0**-16 * (1 + want[4][0])).all()
    assert_attention(got[1:], z[1:], tuple(w[1:] for w in want))


@pytest.mark.parametrize("n", [1, 320])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_eight_times_smaller_keep_their_bits(fp8idx, D, n):
    """A head whose largest element lies in [8, 16) where the unit's lies in
    [128, 256): its elements down to 2^-10 of its largest one are exact."""
    rng = np.random.default_rng(43)
    H = 20
    q, cache, tables = setup(rng, 1, n, H, 1, D, 16, 64, extra=0)
    q[:] = 0
    q[:, :, 0, 0] = 200.0
    q[:, :, 1:, 0] = 8.0
    # (eight significant bits, the last of them set)
    q[:, :, 1:, 1] = 2.0**-7 * (1 + rng.integers(0, 64, (1, n, H - 1)) / 64 + 1 / 128)
    cache[:, 0, : 16 * 2 * D].reshape(-1, 16, 2, D)[:, :, 0] = 0
    codes = rng.integers(0x70, 0x7F, (4, 16))
    cache[:, 0, : 16 * 2 * D].reshape(-1, 16, 2, D)[:, :, 0, 1] = codes
    sc, put = scales_of(cache, 16, D)
    sc[..., 0] = 1.0
    put()
    attend(fp8idx, q, cache, pick(rng, n, 60, 64), tables, 16, 1.0)


@pytest.mark.parametrize("n", [1, 320])
@pytest.mark.parametrize("top", [-80, -40, -10, 0, 40, 100])
def test_heads_as_far_apart_as_bf16_goes(fp8idx, top, n):
    """Heads of 2^127 next to ones of 2^top: keys that are zero where the
    large heads are not leave those a score of 0."""
    rng = np.random.default_rng(44)
    D, H = 64, 20
    q, cache, tables = setup(rng, 1, n, H, 1, D, 16, 64, extra=0)
    q[:, :, 0::2, 32:] = 0
    q[:, :, 0::2, :32] = 2.0**127 * rng.uniform(1, 1.9, (1, n, H // 2, 32))
    q[:, :, 1::2, :32] = 0
    q[:, :, 1::2, 32:] *= 2.0**top
    q[:, :, 3] = 0
    cache[:, 0, : 16 * 2 * D].reshape(-1, 16, 2, D)[:, :, 0, :32] = 0
    attend(fp8idx, q, cache, pick(rng, n, 60, 64), tables, 16, 0.3 * 2.0**-top)
