"""Norms of the heads with the rotation of their positions, on the GPU, against
64-bit numpy.

The error of an output whose terms (x * norm * weight, bias, times cosine and
sine) have the sum of sizes T: its rounding to the type, and in f32 the norm (a
sum of at most 256 squares, a reciprocal root good to 2 units, four products and
sums) and the cosines and sines (2e-9 of their series, 2^-32 turns of their
angle, a few roundings): under 2^-19 T in all (a mean taken off before adds its
own rounding, 2^-20 of the row's largest element)."""
import numpy as np
import pytest
import torch

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


def tolerance(x, terms, y, dtype, norm):
    """Of outputs y (f64)."""
    half = torch.finfo(dtype).eps / 2
    top = np.abs(x).max(-1, keepdims=True)
    spread = x - x.mean(-1, keepdims=True)
    rms = np.sqrt((spread**2).mean(-1, keepdims=True)) + 1e-3
    extra = 2.0**-20 * top / rms if norm == "layer" else 0.0
    tiny = torch.finfo(dtype).smallest_normal * half if dtype == torch.float16 else 1e-35
    return half * np.abs(y) * 1.01 + 2.0**-19 * (terms + extra * np.maximum(terms, 1)) + tiny


def check(fp8idx, T, H, HK, D, dtype, inv_freq, norm=None, affine=True, far=1 << 17, seed=0, interleaved=False, rot_start=0,
          rope_scale=1.0, in_place=False, bias=None, skip=True):
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, far, T).astype(np.int32)
    if skip and T > 3:
        pos[1], pos[-1] = -1, -(2**31)
    x = [torch.from_numpy(3 * rng.standard_normal((T, h, D)).astype(np.float32)).to(dtype).cuda() for h in (H, HK)]
    w = {}
    if norm and affine:
        for n in "qk":
            w[n + "_weight"] = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
            if norm == "layer" if bias is None else bias:
                w[n + "_bias"] = rng.standard_normal(D).astype(np.float32)
    host = [t.double().cpu().numpy() for t in x]
    out = x if in_place else [torch.full_like(t, float("nan")) for t in x]
    f = torch.tensor(inv_freq, dtype=torch.float32)
    fp8idx.head_norm_rope(x[0], x[1] if HK else None, torch.from_numpy(pos).cuda(), f.cuda(), out[0], out[1] if HK else None,
                          norm=norm, interleaved=interleaved, rot_start=rot_start, rope_scale=rope_scale,
                          **{n: torch.from_numpy(a).cuda() for n, a in w.items() if HK or n[0] == "q"})
    torch.cuda.synchronize()
    for n, a, o in zip("qk", host, out):
        if n == "k" and not HK:
            continue
        y, terms = ref.head_norm_rope(a, pos, f.double().numpy(), norm, w.get(n + "_weight"), w.get(n + "_bias"),
                                      interleaved=interleaved, rot_start=rot_start, rope_scale=rope_scale)
        got = o.double().cpu().numpy()
        none = pos < 0
        if in_place:
            assert np.array_equal(got[none], a[none])
        else:
            assert np.isnan(got[none]).all()
        err, tol = np.abs(got - y), tolerance(a, terms, y, dtype, norm)
        bad = ~(err <= tol) & ~none[:, None, None]
        assert not bad.any(), (n, int(bad.sum()), float(err[bad].max()), np.argwhere(bad)[0])


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_whole_heads(fp8idx, D, norm, dtype):
    for T, H, HK in ((1, 1, 0), (5, 32, 8), (33, 7, 1), (700, 3, 3)):
        check(fp8idx, T, H, HK, D, dtype, freqs(D), norm, seed=T)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,start", [(64, 16, 0), (64, 48, 16), (128, 64, 0), (128, 64, 64), (128, 0, 0), (128, 0, 64),
                                         (8, 0, 8), (16, 16, 0), (24, 16, 8), (72, 64, 8), (80, 80, 0), (96, 32, 64),
                                         (192, 64, 128), (256, 16, 240), (248, 48, 104)])
def test_parts_of_heads(fp8idx, D, rot, start, interleaved):
    for norm, dtype in ((None, torch.bfloat16), ("rms", torch.float32), ("layer", torch.float16)):
        check(fp8idx, 40, 5, 2, D, dtype, freqs(rot) if rot else [], norm, interleaved=interleaved, rot_start=start, seed=rot)


@pytest.mark.parametrize("rot", [8, 24, 40, 128])
def test_neighbouring_pairs(fp8idx, rot):
    """Parts that are no multiple of 16 are whole for neighbouring pairs."""
    check(fp8idx, 40, 5, 2, 128, torch.float32, freqs(rot), "rms", interleaved=True, rot_start=128 - rot)


@pytest.mark.parametrize("far", [2, 1000, 1 << 20, 2**31 - 1])
def test_far_positions(fp8idx, far):
    """The angle's whole turns are taken off exactly.  (At 2^31 positions an
    angle has 2^-32 turns of its own, and the 64-bit oracle 2^-22.)"""
    for inv in (freqs(64), [1.0] * 32, [0.1 * i for i in range(32)], [2.0**-30] * 32, [100.0, -3.0] * 16, [0.0] * 32):
        check(fp8idx, 60, 2, 1, 64, torch.float32, inv, far=far if max(inv) <= 1 else min(far, 1 << 20))


def test_scaled_for_long_contexts(fp8idx):
    for kw in (dict(), dict(scaling="linear", factor=8), dict(scaling="ntk", factor=8),
               dict(scaling="yarn", factor=32, original_len=4096)):
        inv, scale = fp8idx.rope_frequencies(64, 10000.0, **kw)
        check(fp8idx, 40, 4, 1, 128, torch.bfloat16, inv.tolist(), "rms", rope_scale=scale, rot_start=64)


@pytest.mark.parametrize("bias", [False, True])
def test_in_place_and_bias(fp8idx, bias):
    for rot, interleaved in ((128, False), (64, False), (128, True)):
        check(fp8idx, 300, 6, 2, 128, torch.bfloat16, freqs(rot), "rms", in_place=True, bias=bias, interleaved=interleaved)


def test_slices_of_one_tensor(fp8idx):
    """Queries and keys as slices of a projection's output, in place, in a
    captured graph; what lies between and behind them stays."""
    rng = np.random.default_rng(1)
    T, H, HK, D = 50, 6, 2, 128
    buf = torch.from_numpy(rng.standard_normal((T + 3, (H + 2 * HK) * D)).astype(np.float32)).to(torch.bfloat16).cuda()
    before = buf.clone()
    q, k = buf[:T, : H * D].view(T, H, D), buf[:T, H * D: (H + HK) * D].view(T, HK, D)
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32)).cuda()
    inv = torch.tensor(freqs(D)).cuda()
    host = before[:T].double().cpu().numpy()
    fp8idx.head_norm_rope(q, k, pos, inv, q, k, norm="rms")
    eager = buf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8idx.head_norm_rope(q, k, pos, inv, q, k, norm="rms")
    buf.copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, eager)
    assert torch.equal(buf[:T, (H + HK) * D:], before[:T, (H + HK) * D:]) and torch.equal(buf[T:], before[T:])
    for at, h in ((0, H), (H * D, HK)):
        x = host[:, at: at + h * D].reshape(T, h, D)
        y, terms = ref.head_norm_rope(x, pos.cpu().numpy(), inv.double().cpu().numpy(), "rms")
        got = buf[:T, at: at + h * D].double().cpu().numpy().reshape(T, h, D)
        assert (np.abs(got - y) <= tolerance(x, terms, y, torch.bfloat16, "rms")).all()


def test_infinities_and_nan_stay_in_their_rows(fp8idx):
    """Without a norm an element reaches itself and the one it is paired with."""
    for rot, interleaved, a, b in ((64, False, 3, 35), (64, True, 6, 7), (32, False, 40, 40)):
        x = torch.ones((4, 2, 64), device="cuda")
        x[1, 1, a] = float("inf")
        x[2, 0, a] = float("nan")
        out = torch.empty_like(x)
        fp8idx.head_norm_rope(x, None, torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor(freqs(rot)).cuda(), out,
                              interleaved=interleaved)
        bad = torch.zeros_like(x, dtype=torch.bool)
        for e in (a, b):
            bad[1, 1, e] = bad[2, 0, e] = True
        assert torch.isfinite(out[~bad]).all() and not torch.isfinite(out[bad]).any()


def test_rows_of_zeros(fp8idx):
    for norm in ("rms", "layer"):
        x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(x, float("nan"))
        fp8idx.head_norm_rope(x, None, torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor(freqs(128)).cuda(), out,
                              norm=norm)
        assert (out == 0).all()


def _turns():
    """2^256 / (2 pi), whole, by Machin's formula for pi."""
    one = 1 << 320

    def atan_inverse(n):
        total = term = one // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    pi = 4 * (4 * atan_inverse(5) - atan_inverse(239))
    return (one << 256) // (2 * pi)


@pytest.mark.parametrize("kind", ["whole", "halves", "pairs"])
def test_cosines_and_sines(fp8idx, kind):
    """(1, 0) and (0, 1) become the cosines and sines themselves: within 2^-23 at
    every position (every step of the f32 series, over all angles, stays within
    1.02e-7; an angle has 2^-32 turns, 1.5e-9, of its own)."""
    rng = np.random.default_rng(37)
    rot = 64
    D = 64 if kind == "whole" else 128
    inv = np.concatenate([freqs(rot)[:16], rng.uniform(0, 1, 8), -rng.uniform(0, 100, 4), [1.0, 60000.0, 2.0**-30, 0.0]])
    inv = inv.astype(np.float32)
    pos = np.concatenate([[0, 1, 2, 2**31 - 1, 2**31 - 2], rng.integers(0, 1 << 17, 200), rng.integers(0, 2**31, 200)])
    pos = pos.astype(np.int32)
    x = torch.zeros((len(pos), 2, D), device="cuda")
    a = np.arange(rot // 2) * 2 if kind == "pairs" else np.arange(rot // 2)
    b = a + 1 if kind == "pairs" else a + rot // 2
    x[:, 0, a] = 1.0
    x[:, 1, b] = 1.0
    out = torch.empty_like(x)
    fp8idx.head_norm_rope(x, None, torch.from_numpy(pos).cuda(), torch.from_numpy(inv).cuda(), out, interleaved=kind == "pairs")
    got = out.double().cpu().numpy()
    per = _turns()
    angle = np.empty((len(pos), len(inv)))
    for i, f in enumerate(inv):
        top, bottom = float(f).as_integer_ratio()
        for t, p in enumerate(pos):
            turn = (int(p) * top * per // bottom) % (1 << 256) / 2.0**256  # (true division of whole numbers, rounded once)
            angle[t, i] = 2 * np.pi * (turn - round(turn))
    c, s = np.cos(angle), np.sin(angle)
    for name, have, want in (("cos", got[:, 0, a], c), ("sin", got[:, 0, b], s), ("-sin", got[:, 1, a], -s), ("cos", got[:, 1, b], c)):
        err = np.abs(have - want)
        assert (err <= 2.0**-23).all(), (name, float(err.max()), np.unravel_index(err.argmax(), err.shape))
