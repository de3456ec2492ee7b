"""The quantising write into a cache whose blocks share a scale, on the GPU, byte
for byte against the definition."""
import numpy as np
import pytest
import torch

from block_cases import filled_blocks
from oracle import serving as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    return m


def same(got, want, bs, D):
    """Codes equal (0 and -0 are one value), scales equal, the rest untouched."""
    at = bs * 2 * D
    values = ref.e4m3_values()
    a, b = values[got[..., :at]], values[want[..., :at]]
    assert np.array_equal(a, b, equal_nan=True), np.argwhere(~((a == b) | (np.isnan(a) & np.isnan(b))))[:5]
    assert np.array_equal(got[..., at: at + 8], want[..., at: at + 8])
    assert np.array_equal(got[..., at + 8:], want[..., at + 8:])


def check(fp8idx, k, v, slots, cache, bs, dtype):
    """k, v f32 arrays, rounded to dtype for both sides."""
    k, v = (torch.from_numpy(np.asarray(x, np.float32)).to(dtype) for x in (k, v))
    d = torch.from_numpy(cache).cuda()
    fp8idx.fp8_paged_block_store(k.cuda(), v.cuda(), torch.from_numpy(np.asarray(slots, np.int32)).cuda(), d)
    torch.cuda.synchronize()
    want = cache.copy()
    ref.store_blocks(want, slots, k.float().numpy(), v.float().numpy(), bs)
    same(d.cpu().numpy(), want, bs, k.shape[-1])
    return want


def rows(rng, T, H, D, spread=1.0):
    return [rng.standard_normal((T, H, D)) * np.exp(spread * rng.standard_normal((T, H, 1))) for _ in range(2)]


def step_slots(rng, held, new, bs, blocks):
    """Slots of a step: request b holds held[b] tokens and gets new[b]."""
    free = iter(rng.permutation(blocks))
    out = []
    for h, n in zip(held, new):
        first = h // bs
        own = [next(free) for _ in range(first, (h + n + bs - 1) // bs if n else first)]
        out += [int(own[p // bs - first]) * bs + p % bs for p in range(h, h + n)]
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_steps(fp8idx, bs, D, dtype):
    """Decode rows, prompt chunks that open, fill and cross blocks, rows that pad
    the step; a second step on top of the first."""
    rng = np.random.default_rng(bs + D)
    held = np.array([0, 5, bs - 1, bs, 3 * bs + 2, bs // 2, 0, 7])
    new = np.array([1, 1, 1, 2, bs + 3, 3 * bs, 2 * bs, 0])
    blocks = int((-(-(new + bs) // bs)).sum()) + 4
    cache = filled_blocks(rng, blocks, 3, bs, D)
    slots = step_slots(rng, held % bs, new, bs, blocks) + [-1] * 5
    k, v = rows(rng, len(slots), 3, D)
    want = check(fp8idx, k, v, slots, cache, bs, dtype)
    ends = np.array(slots)[np.cumsum(new)[new > 0] - 1]  # a token after each request's last, where its block has room
    more = [int(s) + 1 for s in ends if (s + 1) % bs]
    k, v = rows(rng, len(more), 3, D, spread=2.0)
    check(fp8idx, k, v, more, want, bs, dtype)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (3, 40), (100, 1), (700, 2), (3000, 1), (2000, 8)])
def test_sizes(fp8idx, T, H):
    """Few rows and many: windows of one row up to a block's."""
    rng = np.random.default_rng(T + H)
    bs, D = 32, 64
    blocks = T // bs + 3
    cache = filled_blocks(rng, blocks, H, bs, D)
    slots = step_slots(rng, [7], [T], bs, blocks)
    k, v = rows(rng, T, H, D)
    check(fp8idx, k, v, slots, cache, bs, torch.bfloat16)


def test_scales_grow_by_powers_of_two(fp8idx):
    """Tokens one by one, each larger than the ones before, by little and by
    much; also down to blocks whose earlier codes all vanish."""
    rng = np.random.default_rng(3)
    bs, D = 16, 64
    for factor in (1.0, 1.01, 1.5, 2.0, 2.0001, 4.0, 1000.0, 2.0**40):
        cache = np.zeros((2, 1, ref.block_page_bytes(bs, D)), np.uint8)
        size = 2.0**-100 if factor > 2.0**30 else 1e-3
        for t in range(5):
            k, v = rows(rng, 1, 1, D, spread=0.0)
            cache = check(fp8idx, k * size, v * size, [bs + t], cache, bs, torch.float32)
            size *= factor
        scale = cache[1, 0, bs * 2 * D: bs * 2 * D + 8].copy().view(np.float32)
        assert (scale > 0).all()


def test_equal_and_neighbouring_maxima(fp8idx):
    """Growth at its border: a maximum of exactly the scale's reach, of twice it,
    and of the next numbers above both."""
    bs, D = 16, 64
    for top in (1.0, 448.0, 1.5, 3.0):
        for new in (top, np.nextafter(np.float32(top), np.float32(9e9)), 2 * top, np.nextafter(np.float32(2 * top), np.float32(9e9))):
            cache = np.zeros((1, 1, ref.block_page_bytes(bs, D)), np.uint8)
            first = np.linspace(-top, top, 2 * D).reshape(2, 1, D)
            cache = check(fp8idx, first, first[:, :, ::-1], [0, 1], cache, bs, torch.float32)
            x = np.linspace(-0.3, 1, D).reshape(1, 1, D) * np.float32(new)
            x[0, 0, -1] = new
            check(fp8idx, x, -x, [2], cache, bs, torch.float32)


def test_zeros_nan_and_infinities(fp8idx):
    rng = np.random.default_rng(4)
    bs, D = 16, 128
    for dtype in TYPES:
        cache = filled_blocks(rng, 4, 2, bs, D)
        k, v = rows(rng, 3 * bs, 2, D)
        k[5, 0] = 0
        k[bs: 2 * bs] = 0          # a block of zeros: scale 0
        v[:, :, 3] = np.nan
        k[2, 1, 7], k[2, 1, 8], v[9, 0] = np.inf, -np.inf, np.inf
        v[2 * bs:, 1] = np.nan     # a block of NaN alone
        cache = check(fp8idx, k, v, np.arange(3 * bs), cache, bs, dtype)
        # onto blocks with scale 0
        cache = np.array(cache)
        k, v = rows(rng, 3, 2, D)
        check(fp8idx, k, v, [bs + 14, bs + 15, 2 * bs + 15], cache, bs, dtype)
        z = np.zeros((2, 2, D))
        check(fp8idx, z, z, [bs + 3, 3 * bs + 1], cache, bs, dtype)


@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e30, 3e38])
def test_sizes_of_values(fp8idx, size):
    rng = np.random.default_rng(5)
    bs, D = 16, 64
    x = np.clip(rng.standard_normal((bs, 1, D)) / 5, -1, 1) * size
    cache = check(fp8idx, x[:7], -x[:7], np.arange(7), np.zeros((1, 1, ref.block_page_bytes(bs, D)), np.uint8), bs, torch.float32)
    check(fp8idx, x[7:] * min(1.0, 3e38 / size / 1.1), x[7:], np.arange(7, bs), cache, bs, torch.float32)


def test_slots_that_are_skipped(fp8idx):
    rng = np.random.default_rng(6)
    bs, D = 16, 64
    cache = filled_blocks(rng, 5, 2, bs, D)
    n = 5 * bs
    for slots in ([-1, 0, 1, 2, -5, n, n + 1, 2**31 - 1, -(2**31), n - 1], [-1] * 4, [n - 2, n - 1, n], [15, 16, 17, 47, 48],
                  [3, 4, 36, 37, 20, 64], [-1, 0], [31, -1, 32]):
        k, v = rows(rng, len(slots), 2, D)
        check(fp8idx, k, v, slots, cache, bs, torch.bfloat16)


def test_strides_and_replay(fp8idx):
    """Slices of one tensor, caches with space between pages and with heads
    outermost, a captured call replayed."""
    rng = np.random.default_rng(7)
    bs, D, H, T = 32, 128, 2, 90
    blocks = 6
    cache = filled_blocks(rng, blocks, H, bs, D)
    slots = step_slots(rng, [5, 0], [50, 40], bs, blocks)
    k, v = (x.astype(np.float32) for x in rows(rng, T, H, D))
    want = cache.copy()
    kv = torch.empty((T, 2 * H + 1, D + 8), device="cuda")
    kv[:, :H, :D], kv[:, H + 1:, :D] = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    ref.store_blocks(want, slots, k, v, bs)
    page = cache.shape[2]
    wide = torch.full((blocks, H, page + 32), 77, dtype=torch.uint8, device="cuda")
    outer = torch.empty((H, blocks, page), dtype=torch.uint8, device="cuda")
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    for d in (wide[..., :page], outer.transpose(0, 1)):
        d.copy_(torch.from_numpy(cache).cuda())
        fp8idx.fp8_paged_block_store(kv[:, :H, :D], kv[:, H + 1:, :D], s, d)
        same(d.cpu().numpy(), want, bs, D)
        d.copy_(torch.from_numpy(cache).cuda())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fp8idx.fp8_paged_block_store(kv[:, :H, :D], kv[:, H + 1:, :D], s, d)
        for _ in range(2):  # (twice: the scales have what they need)
            graph.replay()
        torch.cuda.synchronize()
        same(d.cpu().numpy(), want, bs, D)
    assert (wide[..., page:] == 77).all()


def test_far_blocks(fp8idx):
    """Blocks more than 2^32 bytes apart."""
    rng = np.random.default_rng(8)
    bs, D, H = 16, 64, 2
    cache = filled_blocks(rng, 4, H, bs, D)
    far, page = 2 << 30, cache.shape[2]
    space = torch.empty(3 * far + H * page, dtype=torch.uint8, device="cuda")
    d = space.as_strided((4, H, page), (far, page, 1))
    d.copy_(torch.from_numpy(cache).cuda())
    k, v = (x.astype(np.float32) for x in rows(rng, 30, H, D))
    slots = list(range(3 * bs, 4 * bs)) + list(range(2 * bs + 1, 2 * bs + 15))
    fp8idx.fp8_paged_block_store(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                                 torch.tensor(slots, dtype=torch.int32, device="cuda"), d)
    ref.store_blocks(cache, slots, k, v, bs)
    same(d.cpu().numpy(), cache, bs, D)
