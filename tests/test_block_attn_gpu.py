"""Dense attention over a cache whose blocks share a scale, on the GPU, against
64-bit numpy (the error bound is derived in block_cases.py)."""
import numpy as np
import pytest
import torch

from block_cases import assert_block_attention, filled_blocks, scales_of, set_scales
from oracle import serving as ref
from serving import bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    m.device_status()
    return m


def setup(rng, ctx, new, H, HK, D, bs, pad_rows=0, spread=0.3, extra=2, max_blocks=None):
    """Inputs of requests with ctx[b] positions, the last new[b] of them rows."""
    ctx, new = np.asarray(ctx), np.asarray(new)
    per = max_blocks or max(1, -(-int(ctx.max()) // bs))
    blocks = len(ctx) * per + extra
    return {"q": bf16(rng.standard_normal((int(new.sum()) + pad_rows, H, D))),
            "cache": filled_blocks(rng, blocks, HK, bs, D, spread),
            "tables": rng.permutation(blocks)[: len(ctx) * per].astype(np.int32).reshape(len(ctx), per),
            "ctx": ctx.astype(np.int32), "cu": np.concatenate([[0], new.cumsum()]).astype(np.int32), "bs": bs}


def call(fp8idx, x, scale, window=0, workspace=None, stream=None, d=None):
    d = d or {n: torch.from_numpy(x[n]).cuda() for n in ("cache", "tables", "ctx", "cu")}
    q = torch.from_numpy(x["q"]).to(torch.bfloat16).cuda()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    fp8idx.fp8_paged_block_attn(q, d["cache"], d["tables"], d["ctx"], d["cu"], scale, out, lse=lse, window=window,
                                workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
    return out, lse


def check(fp8idx, x, scale=None, window=0, what="", **kw):
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    out, lse = call(fp8idx, x, scale, window, **kw)
    want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], x["bs"], scale, window)
    assert_block_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want, what)
    return out, lse


def check_rows(out, lse, want, rows, what=""):
    """Only the rows (or rows and heads) `rows` (a numpy mask) against the figures `want`."""
    o, z = out.float().cpu().numpy()[rows], lse.cpu().numpy()[rows]
    w = [x[rows] for x in want]
    if rows.ndim == 2:
        o, z, w = o[:, None], z[:, None], [x[:, None] for x in w]
    assert_block_attention(o, z, w, what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_block_sizes(fp8idx, bs, D):
    rng = np.random.default_rng(bs + D)
    check(fp8idx, setup(rng, [300, 77, 150], [2, 3, 40], 8, 2, D, bs))


@pytest.mark.parametrize("H,HK", [(1, 1), (2, 2), (7, 1), (15, 3), (16, 2), (17, 1), (32, 1), (33, 1), (64, 1), (65, 1),
                                  (127, 1), (128, 1), (24, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(fp8idx, H, HK, D):
    """One row, two, and more than one unit of 256 rows and heads."""
    rng = np.random.default_rng(H + HK + D)
    check(fp8idx, setup(rng, [200, 290, 19], [1, 2, 9], H, HK, D, 16))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 64, 127, 128, 129, 255, 256, 257, 384, 511, 1000, 2049])
def test_lengths(fp8idx, length):
    rng = np.random.default_rng(length)
    for new in (1, min(length, 5)):
        check(fp8idx, setup(rng, [length], [new], 4, 2, 128, 64), what=f"{new} rows")
    check(fp8idx, setup(rng, [length], [min(length, 70)], 4, 1, 64, 32), what="two tiles of rows")


@pytest.mark.parametrize("new", [8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_row_counts(fp8idx, new):
    """Rows in one copy, two, four and eight, one tile of rows and two, and a
    last unit of every kind."""
    rng = np.random.default_rng(new)
    check(fp8idx, setup(rng, [new + 130], [new], 1, 1, 128, 64))
    check(fp8idx, setup(rng, [new], [new], 2, 2, 64, 16))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 127, 128, 129, 300, 10**6, 2**31 - 1])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(fp8idx, window, D):
    rng = np.random.default_rng(window % 1000 + D)
    check(fp8idx, setup(rng, [700, 40, 333], [3, 40, 80], 6, 2, D, 32), window=window)


def test_mixed_batch_and_empty_requests(fp8idx):
    """Prompt chunks next to decode rows, requests without rows, without
    positions, with more rows than positions, and rows past the last request."""
    rng = np.random.default_rng(5)
    x = setup(rng, [500, 0, 130, 0, 7, 260, 1, 90], [100, 0, 1, 3, 7, 0, 1, 95], 8, 2, 128, 16, pad_rows=9)
    for window in (0, 64):
        check(fp8idx, x, window=window)
    x["cu"] = np.zeros_like(x["cu"])  # no rows at all
    out, lse = call(fp8idx, x, 0.1)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_many_requests(fp8idx):
    """More units than CTAs: none is cut, or every one has a neighbour."""
    rng = np.random.default_rng(6)
    ctx = rng.integers(1, 90, 400)
    check(fp8idx, setup(rng, ctx, np.minimum(ctx, rng.integers(0, 4, 400)), 4, 2, 64, 16))
    x = setup(rng, rng.integers(1, 20, 4096), np.ones(4096, int), 1, 1, 64, 16, extra=0)
    check(fp8idx, x)


@pytest.mark.parametrize("heads", [1, 5])
def test_one_long_request(fp8idx, heads):
    """Every CTA has a piece of the same unit."""
    rng = np.random.default_rng(heads)
    check(fp8idx, setup(rng, [50000], [2], heads, 1, 128, 128))
    check(fp8idx, setup(rng, [30011], [1], heads, 1, 64, 16))


@pytest.mark.parametrize("H,new", [(100, 2), (100, 1), (7, 30), (127, 3), (64, 2), (43, 5), (3, 60)])
def test_units_that_are_cut(fp8idx, H, new):
    """Every kind of unit in pieces: lanes between the heads of the last position
    and a tile's end, one tile of rows and two."""
    rng = np.random.default_rng(H)
    check(fp8idx, setup(rng, [9000, 700], [new, 1], H, 1, 128, 64))
    check(fp8idx, setup(rng, [4000], [new], H, 1, 64, 32), window=3000)


def test_context_past_the_table(fp8idx):
    """Positions past the block table are not attended, by any row."""
    rng = np.random.default_rng(8)
    x = setup(rng, [200, 300], [4, 180], 4, 1, 128, 16)
    x["tables"] = np.ascontiguousarray(x["tables"][:, :9])
    for window in (0, 100, 20):
        check(fp8idx, x, window=window)


def test_blocks_outside_the_cache(fp8idx):
    """Table entries that name no block: their positions are left out; a row may
    be left with none."""
    rng = np.random.default_rng(9)
    x = setup(rng, [300, 100, 64], [3, 100, 2], 4, 2, 128, 16)
    x["tables"][0, ::3] = -1
    x["tables"][0, 4] = x["cache"].shape[0]
    x["tables"][0, 7] = 2**31 - 1
    x["tables"][1, 2] = -(2**31)
    x["tables"][2, :] = -1
    check(fp8idx, x)
    check(fp8idx, x, window=16)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_where_nobody_looks(fp8idx, D):
    """Bytes past a request's positions, later positions of the same tile and
    blocks of no request hold NaN codes and scales."""
    rng = np.random.default_rng(D)
    bs = 32
    x = setup(rng, [75, 40, 160], [30, 1, 150], 4, 2, D, bs)
    owned = np.zeros((x["cache"].shape[0], bs), bool)
    for b, n in enumerate(x["ctx"]):
        for j in range(n):
            owned[x["tables"][b, j // bs], j % bs] = True
    rows = x["cache"][..., : bs * 2 * D].reshape(x["cache"].shape[0], 2, bs, -1)
    rows[~owned[:, None].repeat(2, 1)] = 0x7F
    sc = scales_of(x["cache"], bs, D)
    sc[~owned.any(1)] = np.nan
    set_scales(x["cache"], bs, D, sc)
    check(fp8idx, x)
    want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], bs, D**-0.5)
    # a NaN value and a NaN key at the last position: of the rows only the last one sees them
    for part in (0, 1):
        y = dict(x, cache=x["cache"].copy())
        for b, n in enumerate(y["ctx"]):
            blk, o = y["tables"][b, (n - 1) // bs], (n - 1) % bs
            y["cache"][blk, :, (2 * o + part) * D + 3] = 0xFF if part else 0x7F
        out, lse = call(fp8idx, y, D**-0.5)
        last = np.zeros(out.shape[0], bool)
        last[y["cu"][1:] - 1] = True
        assert torch.isnan(out[torch.from_numpy(last)]).all()
        if part == 0:
            assert torch.isnan(lse[torch.from_numpy(last)]).all()
        check_rows(out, lse, want, ~last)


def test_bad_value_scales(fp8idx):
    """A block whose value scale is NaN or infinite makes the rows that see it
    NaN, and no others; the log-sum-exp does not go by values."""
    rng = np.random.default_rng(12)
    bs, D = 16, 128
    for bad in (np.nan, np.inf):
        x = setup(rng, [200, 90], [3, 60], 4, 1, D, bs)
        sc = scales_of(x["cache"], bs, D)
        want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], bs, D**-0.5)
        sc[x["tables"][1, 4], :, 1] = bad  # positions 64 .. 79 of the second request
        set_scales(x["cache"], bs, D, sc)
        out, lse = call(fp8idx, x, D**-0.5)
        sees = np.zeros(63, bool)
        sees[3:] = np.arange(30, 90) >= 64
        assert torch.isnan(out[torch.from_numpy(sees)]).all()
        check_rows(out, lse, want, ~sees)
        z, sabs = want[1], want[4]
        assert (np.abs(lse.cpu().numpy() - z) <= 2.0**-16 * (1 + sabs)).all()


def test_value_scales_of_zero(fp8idx):
    """Blocks with scale 0 are zeros, whatever their codes, and keep their
    weight; so do rows that see nothing else."""
    rng = np.random.default_rng(13)
    bs, D = 16, 64
    x = setup(rng, [300, 50, 30], [4, 50, 1], 4, 2, D, bs)
    sc = scales_of(x["cache"], bs, D)
    sc[x["tables"][0, 1::2], :, 1] = 0
    sc[x["tables"][1, 0], :, 1] = 0
    sc[x["tables"][2], :, 1] = 0
    sc[x["tables"][1, 2], :, 0] = 0  # keys, too: scores of zero
    set_scales(x["cache"], bs, D, sc)
    check(fp8idx, x)
    check(fp8idx, x, window=10)


@pytest.mark.parametrize("spread", [2.0, 20.0, 60.0])
def test_value_scales_far_apart(fp8idx, spread):
    """Scales between 2^-spread/2 and 2^spread/2 of one another."""
    rng = np.random.default_rng(int(spread))
    bs, D = 16, 128
    x = setup(rng, [600, 130], [2, 40], 4, 2, D, bs)
    sc = scales_of(x["cache"], bs, D)
    sc[..., 1] = np.exp2(rng.uniform(-spread / 2, spread / 2, sc.shape[:2]) - 5)
    set_scales(x["cache"], bs, D, sc)
    check(fp8idx, x)


@pytest.mark.parametrize("size", [2.0**-100, 2.0**-30, 2.0**30, 2.0**90])
def test_value_scales_of_any_size(fp8idx, size):
    rng = np.random.default_rng(3)
    x = setup(rng, [300], [3], 4, 2, 128, 32)
    sc = scales_of(x["cache"], 32, 128)
    sc[..., 1] *= np.float32(size)
    set_scales(x["cache"], 32, 128, sc)
    check(fp8idx, x)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-20, 1.0, 20.0])
def test_softmax_scales(fp8idx, scale):
    rng = np.random.default_rng(4)
    check(fp8idx, setup(rng, [300, 20], [2, 20], 4, 2, 64, 16), scale=scale)
    check(fp8idx, setup(rng, [500], [130], 2, 1, 128, 16), scale=scale)


@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise(fp8idx, rising):
    """Each block's scores lie far above (below) the last one's: the reference
    is raised in every tile, or never again."""
    rng = np.random.default_rng(14)
    bs, D = 16, 128
    for new in (1, 20, 200):
        x = setup(rng, [900], [new], 2, 1, D, bs)
        sc = scales_of(x["cache"], bs, D)
        order = np.arange(x["tables"].shape[1]) if rising else np.arange(x["tables"].shape[1])[::-1]
        sc[x["tables"][0], 0, 0] *= (order * 0.7).astype(np.float32)
        set_scales(x["cache"], bs, D, sc)
        x["q"] = bf16(np.abs(x["q"]))
        codes = x["cache"][..., : bs * 2 * D].reshape(-1, bs, 2, D)
        codes[:, :, 0] &= 0x7F  # positive keys: scores grow with the scale
        check(fp8idx, x)


def test_queries_of_any_size(fp8idx):
    """Rows of zeros, tiny, huge and NaN queries next to ordinary ones."""
    rng = np.random.default_rng(15)
    x = setup(rng, [200], [12], 4, 2, 128, 16)
    x["q"][1] = 0
    x["q"][2, 1] *= 2.0**-90
    x["q"][3, 2] *= 2.0**-30
    x["q"][4, 0, ::2] = 0
    check(fp8idx, x)
    y = dict(x, q=x["q"].copy())
    y["q"][5, 1, 7] = np.nan
    y["q"][6, 3, 0] = np.inf
    out, lse = call(fp8idx, y, 128**-0.5)
    bad = np.zeros((12, 4), bool)
    bad[5, 1] = bad[6, 3] = True
    assert torch.isnan(out[torch.from_numpy(bad)]).all() and torch.isnan(lse[torch.from_numpy(bad)]).all()
    want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], 16, 128**-0.5)
    check_rows(out, lse, want, ~bad)


def test_strides(fp8idx):
    """Rows, heads and outputs that lie apart, caches with space between pages
    and with heads outermost, tables with longer rows; no log-sum-exp."""
    rng = np.random.default_rng(16)
    bs, D, H, HK = 32, 64, 6, 2
    x = setup(rng, [150, 61], [2, 50], H, HK, D, bs)
    want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], bs, 0.125)
    R, page, n = 52, x["cache"].shape[2], x["cache"].shape[0]
    c = torch.from_numpy(x["cache"]).cuda()
    big = torch.full((n, HK, page + 48), 0x7F, dtype=torch.uint8, device="cuda")
    big[..., :page] = c
    outer = torch.empty((HK, n, page), dtype=torch.uint8, device="cuda")
    outer.copy_(c.transpose(0, 1))
    q = torch.from_numpy(x["q"]).to(torch.bfloat16).cuda()
    qkv = torch.full((R, H + 2 * HK, D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :H, :D] = q
    tables = torch.full((2, x["tables"].shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    tables[:, :-3] = torch.from_numpy(x["tables"]).cuda()
    ctx, cu = torch.from_numpy(x["ctx"]).cuda(), torch.from_numpy(x["cu"]).cuda()
    for cache in (big[..., :page], outer.transpose(0, 1)):
        for heads_first in (False, True):
            o = torch.full((H, R, D + 24) if heads_first else (R, H, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
            out = o[..., :D].transpose(0, 1) if heads_first else o[..., :D]
            lse = torch.full((R, H), float("nan"), device="cuda")
            for z in (lse, None):
                fp8idx.fp8_paged_block_attn(qkv[:, :H, :D], cache, tables[:, :-3], ctx, cu, 0.125, out, lse=z)
                torch.cuda.synchronize()
                assert_block_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want)
            assert torch.isnan(o[..., D:]).all()
    # one query for every row
    one = q[:1].expand(R, H, D)
    out = torch.empty((R, H, D), dtype=torch.bfloat16, device="cuda")
    fp8idx.fp8_paged_block_attn(one, c, tables[:, :-3], ctx, cu, 0.125, out)
    full = torch.empty_like(out)
    fp8idx.fp8_paged_block_attn(one.contiguous(), c, tables[:, :-3], ctx, cu, 0.125, full)
    assert torch.equal(out, full)


def test_far_blocks(fp8idx):
    """Blocks more than 2^32 bytes apart."""
    rng = np.random.default_rng(17)
    x = setup(rng, [300], [3], 4, 2, 128, 64, extra=0)
    n, HK, page = x["cache"].shape
    far = 3 << 30
    space = torch.empty((n - 1) * far + HK * page, dtype=torch.uint8, device="cuda")
    cache = space.as_strided((n, HK, page), (far, page, 1))
    cache.copy_(torch.from_numpy(x["cache"]).cuda())
    d = {m: torch.from_numpy(x[m]).cuda() for m in ("tables", "ctx", "cu")}
    check(fp8idx, x, d=dict(d, cache=cache))


def test_workspace_and_repeats(fp8idx):
    """The same bits on every run and whatever the workspace holds; two streams
    with a workspace each; a captured call replayed on other inputs."""
    rng = np.random.default_rng(18)
    x = setup(rng, [3000, 10, 700], [2, 1, 300], 8, 2, 128, 64)
    size = fp8idx.paged_block_attn_workspace(128)
    ws = [torch.full((size,), fill, dtype=torch.uint8, device="cuda") for fill in (0, 0xFF)]
    first = check(fp8idx, x, workspace=ws[0])
    for w in (ws[1], ws[1], None, ws[0]):
        again = call(fp8idx, x, 128**-0.5, workspace=w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    y = setup(rng, [2500, 900], [1, 40], 8, 2, 128, 64)
    alone = call(fp8idx, y, 128**-0.5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = []
    for s, w, z in zip(streams, ws, (x, y)):
        d = {n: torch.from_numpy(z[n]).cuda() for n in ("cache", "tables", "ctx", "cu")}
        q = torch.from_numpy(z["q"]).to(torch.bfloat16).cuda()
        made.append((s, w, d, q, torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, w, d, q, out, lse in made:
            fp8idx.fp8_paged_block_attn(q, d["cache"], d["tables"], d["ctx"], d["cu"], 128**-0.5, out, lse=lse, workspace=w,
                                        stream=s)
    torch.cuda.synchronize()
    for m, want in zip(made, (first, alone)):
        assert torch.equal(m[4], want[0]) and torch.equal(m[5], want[1])
    s, w, d, q, out, lse = made[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8idx.fp8_paged_block_attn(q, d["cache"], d["tables"], d["ctx"], d["cu"], 128**-0.5, out, lse=lse, workspace=w)
    z = setup(rng, [1500, 640, 3001], [290, 3, 9], 8, 2, 128, 64, extra=d["cache"].shape[0] - 3 * 47)
    assert z["cache"].shape == d["cache"].shape and z["tables"].shape == d["tables"].shape
    z["q"] = np.concatenate([z["q"], z["q"][:1]])  # (one row past the last request)
    for n in d:
        d[n].copy_(torch.from_numpy(z[n]))
    q.copy_(torch.from_numpy(z["q"]))
    out.fill_(float("nan"))
    lse.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.block_attention(z["q"].astype(np.float64), z["cache"], z["tables"], z["ctx"], z["cu"], 64, 128**-0.5)
    assert_block_attention(out.float().cpu().numpy(), lse.cpu().numpy(), want)


def test_lengths_that_are_no_prefix_sums(fp8idx):
    """Unspecified rows, but nothing outside the outputs, and no fault."""
    rng = np.random.default_rng(19)
    x = setup(rng, [100, 50, 20], [10, 20, 5], 4, 1, 128, 16)
    guard = torch.full((35 + 64, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.from_numpy(x["q"]).to(torch.bfloat16).cuda()
    cache, tables = torch.from_numpy(x["cache"]).cuda(), torch.from_numpy(x["tables"]).cuda()
    big = 2**31 - 1
    for cu in ([0, 20, 10, 35], [5, 4, 3, 2], [0, 10, 30, 100], [-7, 10, 30, 35], [big, 0, big, 0], [0, big, big, big]):
        for ctx in ([100, 50, 20], [-5, 0, big], [big, big, big]):
            fp8idx.fp8_paged_block_attn(q, cache, tables, torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                                        torch.tensor(cu, dtype=torch.int32, device="cuda"), 0.1, guard[32: 32 + 35])
    torch.cuda.synchronize()
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
    assert torch.isnan(guard[:32]).all() and torch.isnan(guard[-32:]).all()


@pytest.mark.parametrize("handle", [False, True])
def test_own_workspace_on_another_stream(fp8idx, monkeypatch, handle):
    """The workspace that a call allocates belongs to the stream it runs on:
    what the current stream allocates next is other memory."""
    from sparse_attention_fp8_gb300 import _native
    rng = np.random.default_rng(29)
    x = setup(rng, [700, 300], [1, 1], 8, 2, 128, 64)
    d = {n: torch.from_numpy(x[n]).cuda() for n in ("cache", "tables", "ctx", "cu")}
    q = torch.from_numpy(x["q"]).to(torch.bfloat16).cuda()
    out, want = torch.empty_like(q), torch.empty_like(q)
    nbytes = fp8idx.paged_block_attn_workspace(128) + 256
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = []
    monkeypatch.setattr(_native, "_scratch", lambda *a, f=_native._scratch: held.append(w := f(*a)) or w)
    fp8idx.fp8_paged_block_attn(q, d["cache"], d["tables"], d["ctx"], d["cu"], 0.1, out,
                                stream=s.cuda_stream if handle else s)
    used = held.pop().data_ptr()  # (the last reference: the allocator has the memory back)
    other = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != used
    torch.cuda.synchronize()
    fp8idx.fp8_paged_block_attn(q, d["cache"], d["tables"], d["ctx"], d["cu"], 0.1, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and fp8idx.device_status() == fp8idx.FP8IDX_OK


def test_negative_value_scales(fp8idx):
    """A value scale below zero, which no store writes, counts as no number."""
    rng = np.random.default_rng(30)
    x = setup(rng, [256, 200], [1, 40], 4, 2, 128, 32)
    scales = scales_of(x["cache"], 32, 128).copy()
    block = x["tables"][0, 3]
    scales[block, 1, 1] *= -1
    set_scales(x["cache"], 32, 128, scales)
    out, lse = call(fp8idx, x, 0.1)
    scales[block, 1, 1] *= -1
    set_scales(x["cache"], 32, 128, scales)
    want = ref.block_attention(x["q"].astype(np.float64), x["cache"], x["tables"], x["ctx"], x["cu"], 32, 0.1, 0)
    hit = np.zeros(x["q"].shape[:2], bool)
    hit[0, 2:] = True  # (the heads of key head 1, in the request that has the block)
    assert torch.isnan(out[0, 2:]).all()
    check_rows(out, lse, want, ~hit)
    assert np.abs(lse.cpu().numpy() - want[1])[hit].max() < 2.0**-16 * (1 + want[4][hit]).max()


@pytest.mark.parametrize("size", [1e-45, 1e-42, 1e30, 3e38])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_where_nobody_looks(fp8idx, D, size):
    """Scales of blocks that no row sees may be any number: table entries past a
    request's positions (in a tile with seen ones, first and only or last) and
    before a window, with seen blocks of scale 0 in the same tiles and without."""
    rng = np.random.default_rng(31)
    bs = 16
    ctx, new = [75, 300, 20, 700], [30, 2, 1, 200]
    for window in (0, 40):
        x = setup(rng, ctx, new, 4, 2, D, bs, max_blocks=50)
        seen = np.zeros(x["cache"].shape[0], bool)
        for b, (n, m) in enumerate(zip(ctx, new)):
            seen[x["tables"][b, (max(n - m - window + 1, 0) if window else 0) // bs: -(-n // bs)]] = True
        sc = scales_of(x["cache"], bs, D)
        sc[~seen] = size
        for zeros in (False, True):
            if zeros:
                for b in (1, 3):
                    sc[x["tables"][b, (ctx[b] - 1) // bs], :, 1] = 0
            set_scales(x["cache"], bs, D, sc)
            check(fp8idx, x, window=window, what=f"window {window}, zeros {zeros}")


@pytest.mark.parametrize("far", [2.0**-64, 2.0**-63, 2.0**63, 2.0**64])
@pytest.mark.parametrize("new", [1, 40, 130])
def test_value_scales_of_zero_beside_far_ones(fp8idx, new, far):
    """Blocks of scale 0 keep their weight (every score is the same) next to
    scales at the far end of the range, before them and after them."""
    rng = np.random.default_rng(32)
    bs, D = 16, 128
    x = setup(rng, [560], [new], 2, 1, D, bs)
    sc = scales_of(x["cache"], bs, D)
    sc[..., 0] = 0
    sc[..., 1] = 1
    table = x["tables"][0]
    sc[table[8:16], :, 1] = far  # the second tile
    sc[table[[3, 9, 11, 18, 30]], :, 1] = 0
    set_scales(x["cache"], bs, D, sc)
    check(fp8idx, x)
    check(fp8idx, x, window=200)


def test_value_scales_farther_apart_than_the_range(fp8idx):
    """A block of tiny values (a scale that a store of them writes) next to
    ordinary ones: its values do not count, its weights do."""
    rng = np.random.default_rng(33)
    bs, D = 16, 128
    for new in (1, 40, 130):
        x = setup(rng, [560], [new], 2, 1, D, bs)
        sc = scales_of(x["cache"], bs, D)
        sc[x["tables"][0, [2, 9, 20]], :, 1] = [[1e-42], [1e-45], [2e-38]]
        set_scales(x["cache"], bs, D, sc)
        check(fp8idx, x)


@pytest.mark.parametrize("size", [1e-38, 1e36, 3e38])
def test_value_scales_at_the_ends_of_f32(fp8idx, size):
    """Whole units and units in pieces, whose sums are larger than their means."""
    rng = np.random.default_rng(38)
    bs, D = 32, 128
    for ctx, new in ((100, 1), (3000, 2), (3000, 130)):
        x = setup(rng, [ctx], [new], 2, 1, D, bs)
        codes = x["cache"][..., : bs * 2 * D].reshape(-1, bs, 2, D)
        codes[:, :, 1] = codes[:, :, 1] & 0x87 | 0x30  # values of 0.5 to 0.94
        sc = scales_of(x["cache"], bs, D)
        sc[..., 0] = 0.01
        sc[..., 1] = size
        set_scales(x["cache"], bs, D, sc)
        out, _ = check(fp8idx, x, what=f"{ctx} positions, {new} rows")
        assert (out.abs() > 0).any()


@pytest.mark.parametrize("size", [1e-38, 1.0, 3e38])
@pytest.mark.parametrize("D", [64, 128])
def test_first_tiles_without_values(fp8idx, D, size):
    """Value scales of any size after tiles whose blocks all have scale 0, in
    either group's tiles."""
    rng = np.random.default_rng(34)
    bs = 32
    for ctx, new, zeros in ((200, 1, 4), (300, 1, 4), (300, 1, 8), (513, 3, 12), (300, 130, 4), (700, 260, 8), (140, 140, 4)):
        x = setup(rng, [ctx], [new], 2, 1, D, bs)
        codes = x["cache"][..., : bs * 2 * D].reshape(-1, bs, 2, D)
        codes[:, :, 1] = codes[:, :, 1] & 0x87 | 0x30  # values of 0.5 to 0.94
        sc = scales_of(x["cache"], bs, D)
        sc[..., 0] = 0.01
        sc[..., 1] = size
        sc[x["tables"][0, :zeros], :, 1] = 0
        set_scales(x["cache"], bs, D, sc)
        check(fp8idx, x, what=f"{ctx} positions, {new} rows")


@pytest.mark.parametrize("softmax_scale", [0.1, 1.0, -1.0])
def test_negative_key_scales(fp8idx, softmax_scale):
    """A key is code * scale whatever the scale's sign."""
    rng = np.random.default_rng(35)
    bs, D = 16, 128
    for new in (1, 20, 200):
        x = setup(rng, [900], [new], 2, 1, D, bs)
        sc = scales_of(x["cache"], bs, D)
        sc[rng.random(sc.shape[0]) < 0.5, :, 0] *= -1
        set_scales(x["cache"], bs, D, sc)
        check(fp8idx, x, scale=softmax_scale)
        sc[..., 0] = -np.abs(sc[..., 0])
        set_scales(x["cache"], bs, D, sc)
        check(fp8idx, x, scale=softmax_scale)


@pytest.mark.parametrize("ctx,window", [(2**31 - 389, 300), (2**31 - 384, 100), (2**31 - 1, 700), (2**31 - 700, 2000)])
def test_positions_near_two_to_the_31(fp8idx, ctx, window):
    """The last positions that a table may hold, and a row's position past them:
    the same as at the start, with as many blocks less."""
    rng = np.random.default_rng(36)
    bs, D, blocks = 128, 128, 24
    per = 2**24 - 3  # 2^31 - 384 positions
    less = per - blocks
    x = setup(rng, [blocks * bs], [3], 4, 2, D, bs)
    tables = torch.zeros((1, per), dtype=torch.int32, device="cuda")
    tables[:, less:] = torch.from_numpy(x["tables"]).cuda()
    d = {"cache": torch.from_numpy(x["cache"]).cuda(), "tables": tables,
         "ctx": torch.tensor([ctx], dtype=torch.int32, device="cuda"), "cu": torch.from_numpy(x["cu"]).cuda()}
    x["ctx"] = np.array([ctx - less * bs])
    check(fp8idx, x, window=window, d=d)


@pytest.mark.parametrize("window", [2**31, 2**32 + 5, 2**63 - 1])
def test_windows_past_32_bits(fp8idx, window):
    """A window longer than every context is none."""
    rng = np.random.default_rng(39)
    x = setup(rng, [300, 40], [2, 40], 4, 2, 128, 32)
    with_window, without = call(fp8idx, x, 0.1, window=window), call(fp8idx, x, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(with_window, without))


def test_small_query_elements(fp8idx):
    """Elements down to 2^-9 of their head's largest one are exact, smaller ones
    off by 2^-17 of it at most: the score of a key that takes one element."""
    bs, D = 16, 64
    tops = np.array([1.0, 1.9921875, 0.75, 2.0**20, 1.9921875 * 2.0**-40], np.float32)  # (255 / 128 has all of bf16's bits)
    down = np.arange(0, 24)
    bits = np.array([1.0, 129 / 128, 171 / 128, 255 / 128])
    small = (tops[:, None, None] * np.exp2(-down)[:, None] * bits).reshape(len(tops), -1)
    small = bf16(np.minimum(small, tops[:, None]))
    H = small.shape[1]
    q = np.zeros((len(tops), H, D), np.float32)
    q[:, :, 0] = tops[:, None]
    q[:, :, 1] = small
    cache = np.zeros((1, 1, ref.block_page_bytes(bs, D)), np.uint8)
    cache[0, 0, 1] = 0x38  # key element 1 is 1
    set_scales(cache, bs, D, np.ones((1, 1, 2)))
    for r, top in enumerate(tops):
        x = {"q": q[r: r + 1], "cache": cache, "tables": np.zeros((1, 1), np.int32), "ctx": np.array([1], np.int32),
             "cu": np.array([0, 1], np.int32), "bs": bs}
        scale = 2.0**8 / float(top)
        _, lse = call(fp8idx, x, scale)
        got, want = lse[0].double().cpu().numpy(), scale * small[r].astype(np.float64)
        exact = small[r] >= top * 2.0**-9
        assert exact.any() and not exact.all()
        # (scores to 2^8 in f32, the exponential and the logarithm)
        tol = 2.0**-21 * np.maximum(want, 1) + np.where(exact, 0, 2.0**-17 * 2.0**8)
        assert (np.abs(got - want) <= tol).all(), (top, np.abs(got - want).max())
