"""The attention over selected positions on the GPU against 64-bit numpy
(the error bound is derived in serving.py)."""
import numpy as np
import pytest
import torch

from oracle import serving as ref
from serving import assert_attention, bf16, filled_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    m.device_status()
    return m


def pick(rng, n, k, length):
    """k entries: distinct positions in order, then -1."""
    idx = np.full((n, k), -1, np.int32)
    for r in range(n):
        m = min(k, length)
        idx[r, :m] = np.sort(rng.permutation(length)[:m])
    return idx


def decode(fp8idx, q, cache, idx, tables, bs, scale, ctas=0, what=""):
    """q [B, n, H, D] f32, rounded to bf16 for both sides."""
    q = bf16(q)
    B, n, H, D = q.shape
    out = torch.full((B, n, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B * n, H), float("nan"), device="cuda")
    opt = fp8idx.Options(num_ctas=ctas) if ctas else None
    fp8idx.fp8_paged_sparse_attn(torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(),
                                 torch.from_numpy(idx).cuda(), torch.from_numpy(tables).cuda(), scale, out, lse=lse,
                                 options=opt)
    torch.cuda.synchronize()
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
    want = ref.sparse_attention(q.reshape(B * n, H, D).astype(np.float64), cache, idx, tables, bs, scale, next_n=n)
    assert_attention(out.float().cpu().numpy().reshape(B * n, H, D), lse.cpu().numpy(), want, what)
    return out, lse


def setup(rng, B, n, H, HK, D, bs, length, extra=3, spread=0.3):
    blocks = -(-length // bs)
    cache = filled_cache(rng, B * blocks + extra, HK, bs, D, spread)
    tables = rng.permutation(B * blocks + extra)[: B * blocks].astype(np.int32).reshape(B, blocks)
    q = bf16(rng.standard_normal((B, n, H, D)))
    return q, cache, tables


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [1, 16, 32, 64, 128])
def test_decode_block_sizes(fp8idx, bs, D):
    rng = np.random.default_rng(bs + D)
    q, cache, tables = setup(rng, 2, 2, 8, 1, D, bs, 300)
    decode(fp8idx, q, cache, pick(rng, 4, 200, 300), tables, bs, D**-0.5)


@pytest.mark.parametrize("H,HK", [(1, 1), (2, 2), (7, 1), (15, 3), (16, 2), (17, 1), (32, 1), (33, 1), (64, 1), (65, 1),
                                  (128, 1), (96, 3), (24, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_head_layouts(fp8idx, H, HK, D):
    rng = np.random.default_rng(H + HK)
    q, cache, tables = setup(rng, 1, 2, H, HK, D, 16, 400)
    decode(fp8idx, q, cache, pick(rng, 2, 300, 400), tables, 16, D**-0.5)


@pytest.mark.parametrize("k", [1, 2, 31, 127, 128, 129, 255, 256, 257, 640, 1000, 2047, 2048])
def test_decode_lengths_and_splits(fp8idx, k):
    rng = np.random.default_rng(k)
    q, cache, tables = setup(rng, 1, 2, 6, 1, 128, 64, 2100)
    idx = pick(rng, 2, k, 2100)
    for ctas in (0, 1, 2, 4, 8):
        decode(fp8idx, q, cache, idx, tables, 64, 0.1, ctas=ctas, what=f"{ctas} CTAs")


def test_short_contexts_and_empty_rows(fp8idx):
    """Entries of -1 behind, between and in place of the positions."""
    rng = np.random.default_rng(11)
    q, cache, tables = setup(rng, 3, 2, 8, 2, 128, 16, 700)
    idx = pick(rng, 6, 600, 500)
    idx[0] = -1                              # no entry
    idx[1] = -1
    idx[1, 0] = 0                            # one
    idx[2, rng.random(600) < 0.5] = -1       # gaps
    idx[3, :300] = -1                        # whole tiles in front
    idx[4, 130:] = -1
    idx[5] = -1
    idx[5, 599] = 499                        # the last one only
    for ctas in (0, 1, 2, 8):
        decode(fp8idx, q, cache, idx, tables, 16, 0.09, ctas=ctas, what=f"{ctas} CTAs")


def test_bad_entries_are_not_selected(fp8idx):
    """Positions past the table and blocks that are not in the cache."""
    rng = np.random.default_rng(12)
    q, cache, tables = setup(rng, 2, 1, 4, 1, 64, 16, 320)
    idx = pick(rng, 2, 200, 320)
    idx[0, 5], idx[0, 6], idx[1, 7] = 320, 2**31 - 1, -(2**31)
    tables[0, 3], tables[1, 2], tables[1, 5] = -1, cache.shape[0], 2**31 - 1
    decode(fp8idx, q, cache, idx, tables, 16, 0.125)


def test_unselected_bytes_do_not_matter(fp8idx):
    """NaN codes and scales in every row that no entry names."""
    rng = np.random.default_rng(13)
    D, bs = 128, 16
    q, cache, tables = setup(rng, 1, 1, 4, 1, D, bs, 160)
    idx = np.full((1, 140), -1, np.int32)
    idx[0, :70] = np.sort(rng.permutation(160)[:70])
    used = {(int(tables[0, i // bs]), i % bs) for i in idx[0, :70].tolist()}
    for b in range(cache.shape[0]):
        for o in range(bs):
            if (b, o) not in used:
                cache[b, 0, o * 2 * D: (o + 1) * 2 * D] = 0x7F
                cache[b, 0, bs * 2 * D + 8 * o: bs * 2 * D + 8 * o + 8] = 0xFF
    decode(fp8idx, q, cache, idx, tables, bs, D**-0.5)


def test_repeated_entries_and_any_order(fp8idx):
    rng = np.random.default_rng(14)
    q, cache, tables = setup(rng, 1, 2, 8, 1, 128, 64, 500)
    idx = rng.integers(0, 500, (2, 400)).astype(np.int32)
    idx[0, :] = 17                            # one token 400 times
    decode(fp8idx, q, cache, idx, tables, 64, 0.1)


@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_one_dominant_score(fp8idx, where):
    """One score far above the others: their probabilities lie at the end of
    the e4m3 range, and the running maximum jumps where it is met."""
    rng = np.random.default_rng(15)
    D, k = 128, 1024
    q, cache, tables = setup(rng, 1, 1, 5, 1, D, 64, k, extra=0, spread=0.0)
    q[:] = np.abs(q) + 0.5
    at = {"first": 0, "last": k - 1, "middle": 517}[where]
    b, o = int(tables[0, at // 64]), at % 64
    codes, _ = ref.quantise_rows(np.ones((1, D)))
    cache[b, 0, o * 2 * D: o * 2 * D + D] = codes[0]
    for gain in (0.02, 0.1, 1.0, 30.0):
        cache[b, 0, 64 * 2 * D + 8 * o: 64 * 2 * D + 8 * o + 4] = np.array([gain], np.float32).view(np.uint8) 
        decode(fp8idx, q, cache, np.arange(k, dtype=np.int32)[None], tables, 64, D**-0.5, what=f"gain {gain}")


def test_rising_scores(fp8idx):
    """Every tile's maximum is above the last one's."""
    rng = np.random.default_rng(16)
    D, k = 64, 1500
    q, cache, tables = setup(rng, 1, 2, 9, 1, D, 16, k, extra=0, spread=0.0)
    sc = cache[..., 16 * 2 * D:].copy().view(np.float32).reshape(cache.shape[0], 16, 2)
    order = np.empty((cache.shape[0], 16))
    for i in range(k):
        order[tables[0, i // 16], i % 16] = i / k
    sc[..., 0] *= np.exp(4 * order)
    cache[..., 16 * 2 * D:] = sc.reshape(cache.shape[0], 1, -1).view(np.uint8)
    for ctas in (1, 4):
        decode(fp8idx, q, cache, np.tile(np.arange(k, dtype=np.int32), (2, 1)), tables, 16, D**-0.5, ctas=ctas)


def test_value_scales_far_apart(fp8idx):
    rng = np.random.default_rng(17)
    q, cache, tables = setup(rng, 2, 1, 6, 1, 128, 64, 700, spread=3.0)
    idx = pick(rng, 2, 640, 700)
    for ctas in (1, 2):
        decode(fp8idx, q, cache, idx, tables, 64, 0.01, ctas=ctas)


def test_scales_of_either_sign(fp8idx):
    """A cache that another writer filled: key and value scales below 0."""
    rng = np.random.default_rng(27)
    D, bs = 128, 16
    q, cache, tables = setup(rng, 2, 1, 6, 1, D, bs, 700)
    sc = cache[..., bs * 2 * D:].copy().view(np.float32)
    sc *= rng.choice([-1, 1], sc.shape).astype(np.float32)
    cache[..., bs * 2 * D:] = sc.view(np.uint8)
    idx = pick(rng, 2, 640, 700)
    for ctas in (0, 1, 2):
        decode(fp8idx, q, cache, idx, tables, bs, 0.09, ctas=ctas)


def test_selected_nan_reaches_its_row_alone(fp8idx):
    """A NaN key, value or scale makes the rows that select it NaN, and no
    other row."""
    rng = np.random.default_rng(28)
    D, bs = 128, 16
    q, cache, tables = setup(rng, 1, 6, 4, 1, D, bs, 400)
    idx = np.stack([np.arange(5, 305), np.arange(100, 400)] * 3).astype(np.int32)
    bad = cache.copy()
    for at, lo, value in ((0, 0, 0x7F), (1, D, 0x7F), (2, None, 0xFF), (3, None, 0xFF)):  # tokens 0 .. 3
        b = tables[0, 0]
        if lo is not None:
            bad[b, 0, at * 2 * D + lo] = value
        else:
            o = bs * 2 * D + 8 * at + (4 if at == 3 else 0)
            bad[b, 0, o: o + 4] = value
    out, _ = decode(fp8idx, q, bad, idx, tables, bs, 0.09)
    for at in range(4):
        one = idx.copy()
        one[2, 0] = at
        dq = torch.from_numpy(bf16(q)).to(torch.bfloat16).cuda()
        got = torch.empty_like(dq)
        fp8idx.fp8_paged_sparse_attn(dq, torch.from_numpy(bad).cuda(), torch.from_numpy(one).cuda(),
                                     torch.from_numpy(tables).cuda(), 0.09, got)
        others = [0, 1, 3, 4, 5]
        assert torch.equal(got[:, others], out[:, others]), at
        hit = got[0, 2].isnan()
        assert (hit[:, 0].all() and hit.sum() == 4) if at == 1 else hit.all(), at


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, 3.0])
def test_softmax_scales(fp8idx, scale):
    rng = np.random.default_rng(18)
    q, cache, tables = setup(rng, 1, 1, 4, 1, 128, 64, 300)
    decode(fp8idx, q, cache, pick(rng, 1, 290, 300), tables, 64, scale)


def test_query_sizes(fp8idx):
    """Zero queries, tiny and huge ones, heads of very different size."""
    rng = np.random.default_rng(19)
    q, cache, tables = setup(rng, 4, 1, 6, 1, 128, 16, 256)
    q[0] = 0
    q[1] = bf16(q[1] * 1e-20)
    q[2] = bf16(q[2] * 1e4)
    q[3] = bf16(q[3] * np.array([1e-6, 1e-3, 1, 1, 10, 100]).reshape(1, 6, 1))
    cache2 = cache.copy()
    idx = pick(rng, 4, 200, 256)
    decode(fp8idx, q, cache2, idx, tables, 16, 1e-3)


@pytest.mark.parametrize("n", [2, 320])
def test_heads_of_far_apart_sizes(fp8idx, n):
    """The heads' query rows differ by up to 2^20: each keeps its own bits
    (a cluster per row, and persistent CTAs)."""
    rng = np.random.default_rng(33)
    q, cache, tables = setup(rng, 1, n, 20, 1, 64, 16, 200)
    q[:, ::2] *= np.exp2(rng.integers(-16, 5, (1, (n + 1) // 2, 20, 1)))
    q[:, :, 7] = 0
    decode(fp8idx, q, cache, pick(rng, n, 150, 200), tables, 16, 0.125)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_query_without_a_value_spoils_its_head_alone(fp8idx, value):
    rng = np.random.default_rng(29)
    q, cache, tables = setup(rng, 2, 1, 6, 1, 128, 16, 256)
    q[1, 0, 2] = 0
    idx = pick(rng, 2, 200, 256)
    want, _ = decode(fp8idx, q, cache, idx, tables, 16, 0.09)
    dq = torch.from_numpy(bf16(q)).to(torch.bfloat16).cuda()
    dq[1, 0, 2, 77] = value
    got = torch.empty_like(dq)
    fp8idx.fp8_paged_sparse_attn(dq, torch.from_numpy(cache).cuda(), torch.from_numpy(idx).cuda(),
                                 torch.from_numpy(tables).cuda(), 0.09, got)
    assert got[1, 0, 2].isnan().all()
    got[1, 0, 2] = want[1, 0, 2]
    assert torch.equal(got, want)


def prefill(fp8idx, q, cache, idx, tables, cu, bs, scale, what=""):
    q = bf16(q)
    M, H, D = q.shape
    out = torch.full((M, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((M, H), float("nan"), device="cuda")
    fp8idx.fp8_mqa_sparse_attn_paged(torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(),
                                     torch.from_numpy(tables).cuda(), torch.from_numpy(cu).cuda(),
                                     torch.from_numpy(idx).cuda(), scale, out, lse=lse)
    torch.cuda.synchronize()
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
    want = ref.sparse_attention(q.astype(np.float64), cache, idx, tables, bs, scale, cu_seq_lens=cu)
    assert_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want, what)


@pytest.mark.parametrize("D,bs", [(128, 64), (64, 16), (128, 1)])
def test_prefill(fp8idx, D, bs):
    """Requests of uneven length (one of none), rows that select in their own
    request, in two, and past the last column."""
    rng = np.random.default_rng(20 + D)
    lens = np.array([70, 0, 333, 1, 200])
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    blocks = -(-333 // bs)
    cache = filled_cache(rng, 5 * blocks + 2, 2, bs, D)
    tables = rng.permutation(5 * blocks + 2)[: 5 * blocks].astype(np.int32).reshape(5, blocks)
    M, k = 23, 180
    idx = np.full((M, k), -1, np.int32)
    for r in range(M):
        req = [0, 2, 2, 4, 3][r % 5]
        m = min(k, int(lens[req]))
        idx[r, :m] = np.sort(cu[req] + rng.permutation(int(lens[req]))[:m])
    idx[7] = np.sort(rng.permutation(int(cu[-1]))[:k])   # columns of several requests
    idx[8, :5] = cu[-1], cu[-1] + 7, 2**31 - 1, -1, cu[-1] - 1
    q = bf16(rng.standard_normal((M, 10, D)))
    prefill(fp8idx, q, cache, idx, tables, cu, bs, D**-0.5)


@pytest.mark.parametrize("cu", [[-(2**31), 400], [-5, 100], [300, 200], [2**31 - 1, -(2**31)], [0, 2**31 - 1]])
def test_prefill_lengths_that_are_no_prefix_sums(fp8idx, cu):
    """Columns whose place would lie outside the request's table select
    nothing (the call reads nothing outside of it)."""
    rng = np.random.default_rng(34)
    cache = filled_cache(rng, 12, 1, 16, 64)
    tables = rng.permutation(12).astype(np.int32).reshape(1, 12)
    cu = np.array(cu, np.int64)
    idx = np.sort(rng.integers(0, 400, (3, 150)), axis=1).astype(np.int32)
    q = bf16(rng.standard_normal((3, 4, 64)))
    out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 4), device="cuda")
    fp8idx.fp8_mqa_sparse_attn_paged(torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(),
                                     torch.from_numpy(tables).cuda(), torch.from_numpy(cu.astype(np.int32)).cuda(),
                                     torch.from_numpy(idx).cuda(), 0.125, out, lse=lse)
    tok = np.where((idx >= cu[0]) & (idx < cu[1]), idx - cu[0], -1)
    tok = np.where(tok < 12 * 16, tok, -1).astype(np.int32)
    want = ref.sparse_attention(q.astype(np.float64), cache, tok, np.repeat(tables, 3, 0), 16, 0.125, next_n=1)
    assert_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want)


def test_more_rows_than_sms(fp8idx):
    """More units of work than the GPU runs at once, with uneven selections."""
    rng = np.random.default_rng(22)
    lens = np.array([400, 300])
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cache = filled_cache(rng, 60, 2, 16, 64)
    tables = rng.permutation(60)[:50].astype(np.int32).reshape(2, 25)
    M, k = 700, 150
    idx = np.full((M, k), -1, np.int32)
    for r in range(M):
        req = int(r >= 350)
        m = int(rng.integers(0, k + 1))
        idx[r, :m] = np.sort(cu[req] + rng.permutation(int(lens[req]))[:m])
    prefill(fp8idx, bf16(rng.standard_normal((M, 6, 64))), cache, idx, tables, cu, 16, 0.125)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [3, 20])
@pytest.mark.parametrize("rows_per_sm,k", [(2, 700), (3, 513), (5, 130), (7, 300)])
def test_several_units_a_cta(fp8idx, D, H, rows_per_sm, k):
    """Odd and even numbers of rows on an SM, one more on some of them, with
    tiles and rows that select nothing among them."""
    rng = np.random.default_rng(rows_per_sm + k + D)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    M, bs, length = rows_per_sm * sms + 37, 32, 900
    cache = filled_cache(rng, 40, 1, bs, D)
    blocks = -(-length // bs)
    tables = rng.permutation(40)[:blocks].astype(np.int32).reshape(1, blocks)
    idx = np.sort(rng.integers(0, length, (M, k)), axis=1).astype(np.int32)
    for r in range(M):
        what = rng.integers(0, 6)
        if what == 0:
            idx[r] = -1
        elif what == 1:
            idx[r, int(rng.integers(0, k)):] = -1
        elif what == 2:
            t = int(rng.integers(0, -(-k // 128)))
            idx[r, 128 * t: 128 * (t + 1)] = -1
    prefill(fp8idx, bf16(rng.standard_normal((M, H, D))), cache, idx, tables, np.array([0, length], np.int32), bs, D**-0.5)


def test_strides(fp8idx):
    """q and out as slices of wider tensors, indices with a longer row
    stride, the cache one layer of a larger one, a sliced block table."""
    rng = np.random.default_rng(23)
    B, n, H, HK, D, bs = 2, 3, 8, 2, 128, 32
    q, cache, tables = setup(rng, B, n, H, HK, D, bs, 300)
    idx = pick(rng, B * n, 250, 300)
    wide_q = torch.randn((B, n, H + 4, 2 * D), device="cuda").to(torch.bfloat16)
    wide_q[:, :, 2: 2 + H, D:] = torch.from_numpy(q).to(torch.bfloat16).cuda()
    layers = torch.randint(0, 256, (cache.shape[0], 3, HK, cache.shape[2]), dtype=torch.uint8, device="cuda")
    layers[:, 1] = torch.from_numpy(cache).cuda()
    wide_i = torch.full((B * n, 300), 7, dtype=torch.int32, device="cuda")
    wide_i[:, 20: 270] = torch.from_numpy(idx).cuda()
    wide_t = torch.full((B, 30), -9, dtype=torch.int32, device="cuda")
    wide_t[:, 3: 3 + tables.shape[1]] = torch.from_numpy(tables).cuda()
    wide_o = torch.full((B, n + 1, H, D + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide_o[:, 1:, :, 1: 1 + D]
    fp8idx.fp8_paged_sparse_attn(wide_q[:, :, 2: 2 + H, D:], layers[:, 1], wide_i[:, 20: 270],
                                 wide_t[:, 3: 3 + tables.shape[1]], 0.1, out)
    torch.cuda.synchronize()
    want = ref.sparse_attention(q.reshape(B * n, H, D).astype(np.float64), cache, idx, tables, bs, 0.1, next_n=n)
    assert_attention(out.float().cpu().numpy().reshape(B * n, H, D), np.where(np.isneginf(want[1]), want[1], want[1]), want)
    assert (wide_o[:, 0] == 5).all() and (wide_o[..., 0] == 5).all() and (wide_o[..., D + 1:] == 5).all()


def test_one_selection_for_all_rows(fp8idx):
    """indices and q as broadcast tensors (row stride 0)."""
    rng = np.random.default_rng(30)
    q, cache, tables = setup(rng, 1, 4, 8, 2, 64, 16, 300)
    idx = pick(rng, 1, 250, 300)
    one = torch.from_numpy(bf16(q[:, :1])).to(torch.bfloat16).cuda()
    out = torch.empty((1, 4, 8, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 8), device="cuda")
    fp8idx.fp8_paged_sparse_attn(one.expand(1, 4, 8, 64), torch.from_numpy(cache).cuda(),
                                 torch.from_numpy(idx).cuda().expand(4, 250), torch.from_numpy(tables).cuda(), 0.125, out,
                                 lse=lse)
    want = ref.sparse_attention(np.repeat(bf16(q[0, :1]), 4, 0).astype(np.float64), cache, np.repeat(idx, 4, 0), tables, 16,
                                0.125, next_n=4)
    assert_attention(out[0].float().cpu().numpy(), lse.cpu().numpy(), want)


def test_captured_and_on_two_streams(fp8idx):
    """A captured call replayed on new inputs, and two calls at once on two
    streams (no shared scratch)."""
    rng = np.random.default_rng(24)
    q, cache, tables = setup(rng, 2, 2, 16, 1, 128, 64, 1200)
    idx = pick(rng, 4, 1024, 1200)
    dq, dc, dt = torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(), torch.from_numpy(tables).cuda()
    di = torch.from_numpy(idx).cuda()
    out = torch.empty_like(dq)
    fp8idx.fp8_paged_sparse_attn(dq, dc, di, dt, 0.1, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8idx.fp8_paged_sparse_attn(dq, dc, di, dt, 0.1, out)
    q2 = bf16(rng.standard_normal(q.shape))
    idx2 = pick(rng, 4, 1024, 700)
    dq.copy_(torch.from_numpy(q2)), di.copy_(torch.from_numpy(idx2))
    g.replay()
    torch.cuda.synchronize()
    first = out.clone()
    want = ref.sparse_attention(q2.reshape(4, 16, 128).astype(np.float64), cache, idx2, tables, 64, 0.1, next_n=2)
    assert_attention(out.float().cpu().numpy().reshape(4, 16, 128), want[1], want)
    outs = [torch.empty_like(dq) for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, o in enumerate(outs):
        fp8idx.fp8_paged_sparse_attn(dq, dc, di, dt, 0.1, o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)  # the same bits every time


def test_long_cache_offsets(fp8idx):
    """Pages whose byte offset passes 32 bits."""
    rng = np.random.default_rng(25)
    D, bs = 128, 64
    page = ref.page_bytes(bs, D)
    blocks = (5 << 30) // page
    dev = torch.zeros((blocks, 1, page), dtype=torch.uint8, device="cuda")
    small = filled_cache(rng, 6, 1, bs, D)
    ids = np.array([0, blocks - 1, blocks // 2, (1 << 32) // page + 1, (1 << 31) // page + 1, 7])
    dev[torch.from_numpy(ids).cuda()] = torch.from_numpy(small).cuda()
    q = bf16(rng.standard_normal((1, 1, 8, D)))
    idx = pick(rng, 1, 300, 6 * bs)
    out = torch.empty((1, 1, 8, D), dtype=torch.bfloat16, device="cuda")
    fp8idx.fp8_paged_sparse_attn(torch.from_numpy(q).to(torch.bfloat16).cuda(), dev, torch.from_numpy(idx).cuda(),
                                 torch.from_numpy(ids.astype(np.int32)[None]).cuda(), 0.1, out)
    want = ref.sparse_attention(q[0].astype(np.float64), small, idx, np.arange(6, dtype=np.int32)[None], bs, 0.1, next_n=1)
    assert_attention(out.float().cpu().numpy()[0], want[1], want)


def test_no_rows(fp8idx):
    cache = torch.zeros((2, 1, fp8idx.kv_page_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    q = torch.empty((0, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    fp8idx.fp8_paged_sparse_attn(q, cache, torch.empty((0, 8), dtype=torch.int32, device="cuda"),
                                 torch.empty((0, 2), dtype=torch.int32, device="cuda"), 1.0, torch.empty_like(q))


def test_outputs_between_inputs_and_in_other_orders(fp8idx):
    """q and out as column ranges of one tensor (their rows lie between one
    another), and an out whose heads lie outermost."""
    rng = np.random.default_rng(31)
    B, n, H, HK, D, bs = 2, 3, 8, 2, 64, 16
    q, cache, tables = setup(rng, B, n, H, HK, D, bs, 300)
    idx = pick(rng, B * n, 250, 300)
    dc, di, dt = (torch.from_numpy(a).cuda() for a in (cache, idx, tables))
    both = torch.full((B, n, H, 3 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    both[..., D: 2 * D] = torch.from_numpy(q).to(torch.bfloat16)
    turned = torch.full((H, B, n, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    want = ref.sparse_attention(bf16(q).reshape(B * n, H, D).astype(np.float64), cache, idx, tables, bs, 0.1, next_n=n)
    for out in (both[..., 2 * D:], turned.permute(1, 2, 0, 3)):
        lse = torch.full((B * n, H), float("nan"), device="cuda")
        fp8idx.fp8_paged_sparse_attn(both[..., D: 2 * D], dc, di, dt, 0.1, out, lse=lse)
        assert_attention(out.float().cpu().numpy().reshape(B * n, H, D), lse.cpu().numpy(), want)
    assert (both[..., :D] == 5).all()


def test_lse_with_strided_arguments(fp8idx):
    """As test_strides, with the log-sum-exp compared."""
    rng = np.random.default_rng(35)
    B, n, H, HK, D, bs = 2, 3, 8, 2, 128, 32
    q, cache, tables = setup(rng, B, n, H, HK, D, bs, 300)
    idx = pick(rng, B * n, 250, 300)
    wide_q = torch.randn((B, n, H + 4, 2 * D), device="cuda").to(torch.bfloat16)
    wide_q[:, :, 2: 2 + H, D:] = torch.from_numpy(q).to(torch.bfloat16).cuda()
    wide_o = torch.full((B, n + 1, H, D + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide_o[:, 1:, :, 1: 1 + D]
    want = ref.sparse_attention(q.reshape(B * n, H, D).astype(np.float64), cache, idx, tables, bs, 0.1, next_n=n)
    for ctas in (0, 1, 2):
        more = torch.full((B * n + 2, H), 7.0, device="cuda")
        lse = more[1:-1]
        fp8idx.fp8_paged_sparse_attn(wide_q[:, :, 2: 2 + H, D:], torch.from_numpy(cache).cuda(), torch.from_numpy(idx).cuda(),
                                     torch.from_numpy(tables).cuda(), 0.1, out, lse=lse,
                                     options=fp8idx.Options(num_ctas=ctas))
        assert_attention(out.float().cpu().numpy().reshape(B * n, H, D), lse.cpu().numpy(), want)
        assert (more[0] == 7).all() and (more[-1] == 7).all()


def test_lse_of_a_replayed_call(fp8idx):
    rng = np.random.default_rng(36)
    q, cache, tables = setup(rng, 2, 2, 16, 1, 128, 64, 1200)
    idx = pick(rng, 4, 1024, 1200)
    dq, dc, dt = torch.from_numpy(q).to(torch.bfloat16).cuda(), torch.from_numpy(cache).cuda(), torch.from_numpy(tables).cuda()
    di = torch.from_numpy(idx).cuda()
    out, lse = torch.empty_like(dq), torch.empty((4, 16), device="cuda")
    fp8idx.fp8_paged_sparse_attn(dq, dc, di, dt, 0.1, out, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8idx.fp8_paged_sparse_attn(dq, dc, di, dt, 0.1, out, lse=lse)
    for length in (700, 3, 1200):
        q2, idx2 = bf16(rng.standard_normal(q.shape)), pick(rng, 4, 1024, length)
        dq.copy_(torch.from_numpy(q2)), di.copy_(torch.from_numpy(idx2))
        out.fill_(float("nan")), lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        want = ref.sparse_attention(q2.reshape(4, 16, 128).astype(np.float64), cache, idx2, tables, 64, 0.1, next_n=2)
        assert_attention(out.float().cpu().numpy().reshape(4, 16, 128), lse.cpu().numpy(), want)


@pytest.mark.parametrize("D,H,rows", [(128, 8, 1), (64, 20, 320)])
def test_lse_and_prompt_rows_past_32_bits_of_offset(fp8idx, D, H, rows):
    rng = np.random.default_rng(37)
    bs = 64
    page = ref.page_bytes(bs, D)
    blocks = (5 << 30) // page
    dev = torch.zeros((blocks, 1, page), dtype=torch.uint8, device="cuda")
    small = filled_cache(rng, 6, 1, bs, D)
    ids = np.array([0, blocks - 1, blocks // 2, (1 << 32) // page + 1, (1 << 31) // page + 1, 7])
    dev[torch.from_numpy(ids).cuda()] = torch.from_numpy(small).cuda()
    q = bf16(rng.standard_normal((rows, H, D)))
    idx = pick(rng, rows, 300, 6 * bs)
    out = torch.empty((rows, H, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((rows, H), device="cuda")
    fp8idx.fp8_mqa_sparse_attn_paged(torch.from_numpy(q).to(torch.bfloat16).cuda(), dev,
                                     torch.from_numpy(ids.astype(np.int32)[None]).cuda(),
                                     torch.tensor([0, 6 * bs], dtype=torch.int32, device="cuda"), torch.from_numpy(idx).cuda(),
                                     0.1, out, lse=lse)
    want = ref.sparse_attention(q.astype(np.float64), small, idx, np.arange(6, dtype=np.int32)[None], bs, 0.1,
                                cu_seq_lens=np.array([0, 6 * bs]))
    assert_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want)
