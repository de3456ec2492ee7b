"""fp8_paged_store on the GPU against the plain definition: the caches are
equal byte for byte (scale and codes follow IEEE f32 arithmetic)."""
import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    return m


def rows(rng, shape):
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape[:-1] + (1,)))
    x[0] = 0.0                         # zeros: scale 0
    if shape[0] > 2:
        x[1] = 0.0
        x[1, ..., 3] = -7.0            # one value
        x[2] *= 1e-6
    return torch.from_numpy(x.astype(np.float32))


def slot_list(rng, T, slots):
    s = rng.permutation(slots)[:T].astype(np.int32)
    s[rng.random(T) < 0.1] = -1
    if T > 4:
        s[3], s[4] = slots, 2**31 - 1  # past the cache: skipped
    return s


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,H,D,bs", [(1, 1, 128, 64), (37, 3, 128, 16), (130, 8, 64, 32), (77, 2, 128, 1), (51, 1, 64, 1),
                                      (300, 5, 64, 128)])
def test_key_value_cache(fp8idx, kind, T, H, D, bs):
    rng = np.random.default_rng(T + D)
    blocks = -(-T // bs) + 3
    k, v = rows(rng, (T, H, D)).to(TYPES[kind]), rows(rng, (T, H, D)).to(TYPES[kind])
    slots = slot_list(rng, T, blocks * bs)
    want = rng.integers(0, 256, (blocks, H, ref.page_bytes(bs, D)), dtype=np.uint8)
    cache = torch.from_numpy(want).cuda()
    assert fp8idx.kv_page_bytes(bs, D) == want.shape[-1]
    fp8idx.fp8_paged_store(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), cache)
    ref.store_kv(want, slots, k.float().numpy(), v.float().numpy(), bs)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,D,bs", [(1, 128, 1), (100, 128, 1), (65, 64, 1), (33, 128, 64), (200, 64, 16), (9, 128, 128)])
def test_index_cache(fp8idx, kind, T, D, bs):
    rng = np.random.default_rng(T + D + 7)
    blocks = -(-T // bs) + 2
    k = rows(rng, (T, D)).to(TYPES[kind])
    slots = slot_list(rng, T, blocks * bs)
    want = rng.integers(0, 256, (blocks, bs * (D + 4)), dtype=np.uint8)
    cache = torch.from_numpy(want).cuda()
    fp8idx.fp8_paged_store(k.cuda(), None, torch.from_numpy(slots).cuda(), cache)
    ref.store_index(want, slots, k.float().numpy(), bs)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_strides(fp8idx):
    """Keys and values as slices of one projection's output, and a cache that
    is one layer of a larger one."""
    rng = np.random.default_rng(3)
    T, H, D, bs, blocks = 45, 2, 128, 16, 5
    x = rows(rng, (T, 3 * H * D)).to(torch.bfloat16).cuda()
    k, v = x[:, H * D: 2 * H * D].unflatten(-1, (H, D)), x[:, 2 * H * D:].unflatten(-1, (H, D))
    page = ref.page_bytes(bs, D)
    whole = rng.integers(0, 256, (blocks, 4, H, page), dtype=np.uint8)
    dev = torch.from_numpy(whole).cuda()
    slots = slot_list(rng, T, blocks * bs)
    fp8idx.fp8_paged_store(k, v, torch.from_numpy(slots).cuda(), dev[:, 2])
    ref.store_kv(whole[:, 2], slots, k.float().cpu().numpy(), v.float().cpu().numpy(), bs)
    assert np.array_equal(dev.cpu().numpy(), whole)
    # heads before blocks
    whole = rng.integers(0, 256, (H, blocks, page), dtype=np.uint8)
    dev = torch.from_numpy(whole).cuda()
    fp8idx.fp8_paged_store(k, v, torch.from_numpy(slots).cuda(), dev.transpose(0, 1))
    ref.store_kv(whole.transpose(1, 0, 2), slots, k.float().cpu().numpy(), v.float().cpu().numpy(), bs)
    assert np.array_equal(dev.cpu().numpy(), whole)


def test_extreme_values(fp8idx):
    """Ties and the edges of the code range: rows whose largest value is a
    power of two (x / scale then meets code midpoints), tiny and huge rows."""
    D = 128
    base = np.linspace(-1, 1, D).astype(np.float32)
    x = np.stack([base * np.float32(f) for f in (448.0, 2.0**-20, 3e38, 1e-30, 1.0, 2.0**100)])
    x[4] = np.tile(np.array([448, 1 / 16 + 1 / 32, -(17 / 16.0), 2.0**-10, 3 * 2.0**-10, 464 / 448, 0, -448], np.float32), 16)
    cache = np.zeros((8, 132), np.uint8)
    dev = torch.from_numpy(cache).cuda()
    slots = np.arange(6, dtype=np.int32)
    fp8idx.fp8_paged_store(torch.from_numpy(x).cuda(), None, torch.from_numpy(slots).cuda(), dev)
    ref.store_index(cache, slots, x, 1)
    assert np.array_equal(dev.cpu().numpy(), cache)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_subnormal_nan_and_infinite_values(fp8idx, dtype):
    """A row of subnormal numbers, one with a NaN (which keeps its place and
    changes no other value), one with an infinity (whose scale is infinite)."""
    D = 64
    rng = np.random.default_rng(5)
    x = torch.from_numpy(np.stack([rng.standard_normal(D) * f for f in (1e-39, 1.0, 1.0, 1.0)]).astype(np.float32)).to(dtype)
    y = x.clone()
    y[1, 5], y[2, 9], y[3, 11] = float("nan"), float("inf"), -float("inf")
    slots = np.arange(4, dtype=np.int32)
    want = np.zeros((4, 68), np.uint8)
    rest = x.float().numpy().copy()
    rest[1, 5] = 0
    ref.store_index(want, slots, rest, 1)
    dev = torch.zeros((4, 68), dtype=torch.uint8, device="cuda")
    fp8idx.fp8_paged_store(y.cuda(), None, torch.from_numpy(slots).cuda(), dev)
    got = dev.cpu().numpy()
    assert np.array_equal(got[0], want[0])
    assert got[1, 5] & 0x7F == 0x7F
    got[1, 5] = want[1, 5]
    assert np.array_equal(got[1], want[1])
    for r, at in ((2, 9), (3, 11)):
        assert np.isposinf(got[r, 64:].view(np.float32)).all()
        assert got[r, at] & 0x7F == 0x7F
        assert (np.delete(got[r, :64], at) & 0x7F == 0).all()


def test_no_tokens_and_capture(fp8idx):
    cache = torch.zeros((4, 64 * 132), dtype=torch.uint8, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    fp8idx.fp8_paged_store(torch.empty((0, 128), device="cuda"), None, none, cache)
    assert not cache.any()
    rng = np.random.default_rng(1)
    k = rows(rng, (20, 128)).cuda()
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    fp8idx.fp8_paged_store(k, None, slots, cache)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8idx.fp8_paged_store(k, None, slots, cache)
    k.copy_(rows(rng, (20, 128)))
    slots.add_(100)
    g.replay()
    torch.cuda.synchronize()
    want = np.zeros((4, 64 * 132), np.uint8)
    ref.store_index(want, np.arange(100, 120), k.cpu().numpy(), 64)
    got = cache.cpu().numpy()
    assert np.array_equal(got[1, 36 * 128: 56 * 128], want[1, 36 * 128: 56 * 128])
    assert np.array_equal(got[1, 64 * 128 + 144: 64 * 128 + 224], want[1, 64 * 128 + 144: 64 * 128 + 224])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_rows_without_a_number_above_zero_keep_their_nan(fp8idx, kind, D):
    """A row of NaN, and NaN among zeros: the maximum is 0, the scale 0, and
    each NaN keeps a NaN code (keys and values, index keys)."""
    H, bs = 2, 16
    x = torch.zeros((4, H, D))
    x[0] = float("nan")
    x[1, :, 5] = float("nan")
    x[2, 0, D - 1] = -float("nan")
    x[3, 1, ::3] = float("nan")
    y = x.flip(0)
    want = np.zeros((2, H, ref.page_bytes(bs, D)), np.uint8)
    slots = np.array([3, 17, 0, 31], np.int32)
    cache = torch.full(want.shape, 0x55, dtype=torch.uint8, device="cuda")
    fp8idx.fp8_paged_store(x.to(TYPES[kind]).cuda(), y.to(TYPES[kind]).cuda(), torch.from_numpy(slots).cuda(), cache)
    got = cache.cpu().numpy()
    index = torch.full((2, bs * (D + 4)), 0x55, dtype=torch.uint8, device="cuda")
    fp8idx.fp8_paged_store(x[:, 0].to(TYPES[kind]).cuda(), None, torch.from_numpy(slots).cuda(), index)
    got_index = index.cpu().numpy()
    for t, s in enumerate(slots.tolist()):
        b, o = divmod(s, bs)
        for part, rows in enumerate((x, y)):
            for h in range(H):
                a = (2 * o + part) * D
                codes, nan = got[b, h, a: a + D], rows[t, h].isnan().numpy()
                assert (codes[nan] & 0x7F == 0x7F).all() and (codes[~nan] == 0).all(), (t, part, h)
                a = bs * 2 * D + 4 * (2 * o + part)
                assert got[b, h, a: a + 4].view(np.float32)[0] == 0
        codes, nan = got_index[b, o * D: (o + 1) * D], x[t, 0].isnan().numpy()
        assert (codes[nan] & 0x7F == 0x7F).all() and (codes[~nan] == 0).all(), t
        assert got_index[b, bs * D + 4 * o: bs * D + 4 * o + 4].view(np.float32)[0] == 0
