"""Refusals of the block-scaled cache's operators and of the head norms (CPU: host
checks with fake pointers that are never dereferenced, before any CUDA call), and
their plain definitions on hand cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_attention_fp8_gb300 as fp8idx
from oracle import serving as ref
from sparse_attention_fp8_gb300 import _native
from test_abi import _t

U8, F32, I32, BF16, F16 = 0, 1, 2, 3, 4
INVALID, UNSUPPORTED = fp8idx.FP8IDX_ERR_INVALID, fp8idx.FP8IDX_ERR_UNSUPPORTED
R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_fp8_gb300 import _build
    _build.build()
    return fp8idx.library()


def refused(lib, st, status, word):
    assert st == status, (st, lib.fp8idx_last_error())
    assert word in lib.fp8idx_last_error(), lib.fp8idx_last_error()


def strided(t, *stride):
    for i, s in enumerate(stride):
        t.stride[i] = s
    return t


def refs(values):
    return [R(v) if isinstance(v, ctypes.Structure) else v for v in values]


def test_sizes(lib):
    for bs in (16, 32, 64, 128):
        for d in (64, 128):
            assert fp8idx.kv_block_page_bytes(bs, d) == ref.block_page_bytes(bs, d)
    assert [fp8idx.kv_block_page_bytes(*a) for a in ((1, 128), (8, 64), (64, 96), (-16, 64))] == [0] * 4
    assert fp8idx.paged_block_attn_workspace(128) > fp8idx.paged_block_attn_workspace(64) > 0
    assert fp8idx.paged_block_attn_workspace(96) == 0


# ---------------------------------------------------------------- head norms
def norm_args(T=6, H=4, HK=2, D=128, rot=128, dtype=BF16, opts=None, **kw):
    at = iter(range(0x100000, 0x900000, 0x10000))
    a = dict(q=_t(dtype, (T, H, D), next(at)), k=_t(dtype, (T, HK, D), next(at)), pos=_t(I32, (T,), next(at)),
             inv=_t(F32, (rot // 2,), next(at)), qw=_t(F32, (D,), next(at)), qb=None, kw=_t(F32, (D,), next(at)), kb=None,
             opts=_native._NormRopeOptions(**{**dict(norm=1, rope_scale=1.0, eps=1e-6), **(opts or {})}),
             oq=_t(dtype, (T, H, D), next(at)), ok=_t(dtype, (T, HK, D), next(at)))
    a.update(kw)
    return refs(a.values()) + [None]


def test_head_norm_rope_refusals(lib):
    f = lib.fp8idx_head_norm_rope
    refused(lib, f(*norm_args(q=None)), INVALID, b"q: null")
    refused(lib, f(*norm_args(dtype=I32)), INVALID, b"q: wrong dtype")
    refused(lib, f(*norm_args(dtype=U8)), INVALID, b"q: wrong dtype")
    refused(lib, f(*norm_args(k=None)), INVALID, b"go together")
    refused(lib, f(*norm_args(ok=None)), INVALID, b"go together")
    refused(lib, f(*norm_args(k=None, ok=None)), INVALID, b"without k")
    refused(lib, f(*norm_args(k=_t(F16, (6, 2, 128)))), INVALID, b"k: wrong dtype")
    refused(lib, f(*norm_args(k=_t(BF16, (5, 2, 128)))), INVALID, b"tokens and head_dim of q")
    refused(lib, f(*norm_args(k=_t(BF16, (6, 2, 64)))), INVALID, b"tokens and head_dim of q")
    refused(lib, f(*norm_args(oq=_t(BF16, (6, 5, 128), 0x900000))), INVALID, b"shape of q")
    refused(lib, f(*norm_args(pos=_t(I32, (5,)))), INVALID, b"positions")
    refused(lib, f(*norm_args(pos=_t(F32, (6,)))), INVALID, b"positions")
    refused(lib, f(*norm_args(inv=_t(I32, (64,)))), INVALID, b"inv_freq")
    refused(lib, f(*norm_args(inv=None)), INVALID, b"inv_freq")
    refused(lib, f(*norm_args(inv=strided(_t(F32, (64,)), 2))), INVALID, b"inv_freq")
    refused(lib, f(*norm_args(qw=_t(F32, (64,)))), INVALID, b"q_weight")
    refused(lib, f(*norm_args(kb=_t(BF16, (128,)))), INVALID, b"k_bias")
    refused(lib, f(*norm_args(opts=dict(norm=0))), INVALID, b"without a norm")
    refused(lib, f(*norm_args(opts=dict(norm=3))), INVALID, b"norm")
    for eps in (-1.0, math.nan, math.inf):
        refused(lib, f(*norm_args(opts=dict(eps=eps))), INVALID, b"eps")
    refused(lib, f(*norm_args(opts=dict(rope_scale=math.nan))), INVALID, b"rope_scale")
    refused(lib, f(*norm_args(D=100, rot=96)), INVALID, b"aligned")
    refused(lib, f(*norm_args(D=264, rot=256)), UNSUPPORTED, b"head_dim")
    refused(lib, f(*norm_args(rot=144)), INVALID, b"outside the head")
    refused(lib, f(*norm_args(rot=64, opts=dict(rot_start=72))), INVALID, b"outside the head")
    refused(lib, f(*norm_args(rot=64, opts=dict(rot_start=-8))), INVALID, b"outside the head")
    refused(lib, f(*norm_args(rot=64, opts=dict(rot_start=4))), UNSUPPORTED, b"rotated elements")
    refused(lib, f(*norm_args(rot=8)), UNSUPPORTED, b"rotated elements")
    refused(lib, f(*norm_args(rot=12, opts=dict(interleaved=1))), UNSUPPORTED, b"rotated elements")
    for name in ("q", "oq"):
        for stride in ((512, 128, 2), (512, 132, 1), (516, 128, 1)):
            refused(lib, f(*norm_args(**{name: strided(_t(BF16, (6, 4, 128), 0x900000), *stride)})), INVALID, b"rows must")
        refused(lib, f(*norm_args(**{name: _t(BF16, (6, 4, 128), 0x900008)})), INVALID, b"aligned")
        refused(lib, f(*norm_args(**{name: strided(_t(BF16, (6, 4, 128), 0x900000), -512, 128, 1)})), INVALID, b"negative")
    refused(lib, f(*norm_args(oq=strided(_t(BF16, (6, 4, 128), 0x900000), 0, 128, 1))), INVALID, b"rows overlap")
    refused(lib, f(*norm_args(oq=strided(_t(BF16, (6, 4, 128), 0x900000), 512, 64, 1))), INVALID, b"rows overlap")
    assert f(*norm_args(T=0)) == fp8idx.FP8IDX_OK


def test_head_norm_rope_overlaps(lib):
    """An output may be its own input and overlap nothing else."""
    f = lib.fp8idx_head_norm_rope
    a = dict(q=_t(BF16, (6, 4, 128), 0x100000), k=_t(BF16, (6, 2, 128), 0x200000), pos=_t(I32, (6,), 0x300000),
             inv=_t(F32, (64,), 0x400000), qw=_t(F32, (128,), 0x500000))
    for at in (0x100010, 0x100000 - 16, 0x200000, 0x200000 - 6 * 4 * 256 + 16, 0x300000 - 16, 0x400000, 0x500000):
        refused(lib, f(*norm_args(**a, oq=_t(BF16, (6, 4, 128), at))), INVALID, b"overlap")
    # the same rows in another order
    refused(lib, f(*norm_args(**a, oq=strided(_t(BF16, (6, 4, 128), 0x100000), 128, 6 * 128, 1))), INVALID, b"overlap")
    for at in (0x100000, 0x200100):
        refused(lib, f(*norm_args(**a, ok=_t(BF16, (6, 2, 128), at))), INVALID, b"overlap")
    refused(lib, f(*norm_args(**a, oq=_t(BF16, (6, 4, 128), 0x600000), ok=_t(BF16, (6, 2, 128), 0x600000 + 256))), INVALID,
            b"overlap")


def test_rope_frequencies():
    inv, scale = fp8idx.rope_frequencies(64)
    assert scale == 1.0 and inv.dtype == torch.float32 and inv.shape == (32,)
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.allclose(inv.numpy(), want, rtol=1e-7)
    assert np.allclose(fp8idx.rope_frequencies(64, scaling="linear", factor=4)[0].numpy(), want / 4, rtol=1e-7)
    ntk = fp8idx.rope_frequencies(64, scaling="ntk", factor=4)[0].numpy()
    assert np.isclose(ntk[0], 1.0) and np.isclose(ntk[-1], want[-1] / 4, rtol=1e-6)  # highest kept, lowest divided
    yarn, scale = fp8idx.rope_frequencies(64, scaling="yarn", factor=16, original_len=4096)
    turns = 4096 * want / (2 * math.pi)
    yarn = yarn.numpy()
    assert np.allclose(yarn[turns > 40], want[turns > 40], rtol=1e-7)
    assert np.allclose(yarn[turns < 0.8], want[turns < 0.8] / 16, rtol=1e-6)
    assert (yarn <= want * 1.0001).all() and (yarn >= want / 16 * 0.9999).all() and (np.diff(yarn) < 0).all()
    assert np.isclose(scale, 0.1 * math.log(16) + 1)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="yarn"), dict(rot_dim=64, scaling="other"), dict(rot_dim=2, scaling="ntk", factor=2),
                dict(rot_dim=64, scaling="yarn", original_len=4096, beta_fast=1.0)):
        with pytest.raises(ValueError):
            fp8idx.rope_frequencies(**bad)


def test_binding_refuses_unknown_norms():
    x = torch.zeros((1, 1, 64))
    with pytest.raises(ValueError, match="norm"):
        fp8idx.head_norm_rope(x, None, x, x, x, norm="batch")


# --------------------------------------------------------------- block store
def store_args(T=5, H=2, D=128, bs=16, blocks=4, dtype=BF16, **kw):
    a = dict(k=_t(dtype, (T, H, D), 0x100000), v=_t(dtype, (T, H, D), 0x200000), slots=_t(I32, (T,), 0x300000),
             kv=_t(U8, (blocks, H, bs * 2 * D + 16), 0x400000))
    a.update(kw)
    return refs(a.values()) + [None]


def test_block_store_refusals(lib):
    f = lib.fp8_paged_block_store
    refused(lib, f(*store_args(k=None)), INVALID, b"k: null")
    refused(lib, f(*store_args(v=None)), INVALID, b"v: null")
    refused(lib, f(*store_args(dtype=U8)), INVALID, b"k: wrong dtype")
    refused(lib, f(*store_args(v=_t(F32, (5, 2, 128)))), INVALID, b"v: wrong dtype")
    refused(lib, f(*store_args(v=_t(BF16, (5, 3, 128)))), INVALID, b"shape of k")
    refused(lib, f(*store_args(slots=_t(I32, (6,)))), INVALID, b"slot_mapping")
    refused(lib, f(*store_args(D=96)), UNSUPPORTED, b"head_dim")
    refused(lib, f(*store_args(bs=8)), UNSUPPORTED, b"block_size")
    refused(lib, f(*store_args(bs=1)), UNSUPPORTED, b"block_size")
    refused(lib, f(*store_args(kv=_t(U8, (4, 2, 16 * 264)))), INVALID, b"fp8idx_kv_block_page_bytes")
    refused(lib, f(*store_args(kv=_t(U8, (4, 2, 16)))), INVALID, b"fp8idx_kv_block_page_bytes")
    refused(lib, f(*store_args(kv=_t(U8, (4, 2, 0)))), INVALID, b"fp8idx_kv_block_page_bytes")
    refused(lib, f(*store_args(kv=_t(U8, (4, 3, 16 * 256 + 16)))), INVALID, b"3 heads")
    refused(lib, f(*store_args(kv=_t(U8, (0, 2, 16 * 256 + 16)))), INVALID, b"empty")
    refused(lib, f(*store_args(kv=_t(U8, (4, 2, 16 * 256 + 16), 0x400008))), INVALID, b"16-byte aligned")
    refused(lib, f(*store_args(kv=_t(I32, (4, 2, 16 * 256 + 16)))), INVALID, b"kv_cache")
    page = 16 * 256 + 16
    for stride in ((2 * page + 8, page, 1), (2 * page, page - 16, 1), (page, page, 1), (2 * page, page, 2)):
        refused(lib, f(*store_args(kv=strided(_t(U8, (4, 2, page), 0x400000), *stride))), INVALID, b"kv_cache")
    refused(lib, f(*store_args(blocks=1 << 27)), UNSUPPORTED, b"2^31")
    for stride in ((256, 128, 2), (260, 128, 1), (256, 132, 1)):
        refused(lib, f(*store_args(v=strided(_t(BF16, (5, 2, 128), 0x200000), *stride))), INVALID, b"rows must")
    for at in (0x100000, 0x200000, 0x300000 - 16):
        refused(lib, f(*store_args(kv=_t(U8, (4, 2, page), at))), INVALID, b"overlap")
    assert f(*store_args(T=0)) == fp8idx.FP8IDX_OK


# ----------------------------------------------------------- block attention
def attn_args(T=5, H=4, HK=2, D=128, bs=16, blocks=9, B=2, mb=3, size=None, ws=0x10000000, scale=0.1, window=0, **kw):
    need = fp8idx.paged_block_attn_workspace(D) or 256
    a = dict(q=_t(BF16, (T, H, D), 0x100000), kv=_t(U8, (blocks, HK, bs * 2 * D + 16), 0x800000), bt=_t(I32, (B, mb), 0x200000),
             ctx=_t(I32, (B,), 0x300000), cu=_t(I32, (B + 1,), 0x400000), scale=scale, window=window,
             out=_t(BF16, (T, H, D), 0x500000), lse=_t(F32, (T, H), 0x600000),
             ws=ctypes.c_void_p(ws) if ws else None, size=ctypes.c_size_t(need if size is None else size))
    a.update(kw)
    return refs(a.values()) + [None]


def test_block_attention_refusals(lib):
    f = lib.fp8_paged_block_attn
    for name in ("q", "kv", "bt", "ctx", "cu", "out"):
        refused(lib, f(*attn_args(**{name: None})), INVALID, b"null")
    refused(lib, f(*attn_args(q=_t(F16, (5, 4, 128)))), INVALID, b"q: wrong dtype")
    refused(lib, f(*attn_args(out=_t(F32, (5, 4, 128)))), INVALID, b"out: wrong dtype")
    refused(lib, f(*attn_args(out=_t(BF16, (5, 5, 128)))), INVALID, b"shape of q")
    refused(lib, f(*attn_args(D=96)), UNSUPPORTED, b"head_dim")
    refused(lib, f(*attn_args(bs=1)), UNSUPPORTED, b"block_size")
    refused(lib, f(*attn_args(HK=3)), INVALID, b"no multiple")
    refused(lib, f(*attn_args(H=258, HK=2)), UNSUPPORTED, b"heads per key head")
    refused(lib, f(*attn_args(H=0, HK=1)), INVALID, b"no heads")
    refused(lib, f(*attn_args(kv=_t(U8, (9, 2, 16 * 264)))), INVALID, b"fp8idx_kv_block_page_bytes")
    refused(lib, f(*attn_args(ctx=_t(I32, (3,)))), INVALID, b"context_lens")
    refused(lib, f(*attn_args(cu=_t(I32, (2,)))), INVALID, b"cu_new_lens")
    refused(lib, f(*attn_args(B=4097)), UNSUPPORTED, b"requests")
    refused(lib, f(*attn_args(bt=strided(_t(I32, (2, 3)), 3, 2))), INVALID, b"block_tables")
    refused(lib, f(*attn_args(mb=(1 << 27) - 16, B=1)), UNSUPPORTED, b"positions")
    refused(lib, f(*attn_args(mb=0)), INVALID, b"empty block table")
    refused(lib, f(*attn_args(window=-1)), INVALID, b"window")
    for scale in (math.nan, math.inf, 3e38):
        refused(lib, f(*attn_args(scale=scale)), INVALID, b"softmax_scale")
    refused(lib, f(*attn_args(lse=_t(F32, (5, 3)))), INVALID, b"lse")
    refused(lib, f(*attn_args(lse=strided(_t(F32, (5, 4)), 5, 1))), INVALID, b"lse")
    refused(lib, f(*attn_args(lse=_t(BF16, (5, 4)))), INVALID, b"lse")
    refused(lib, f(*attn_args(ws=0)), INVALID, b"workspace")
    refused(lib, f(*attn_args(ws=0x10000080)), INVALID, b"workspace")
    refused(lib, f(*attn_args(size=fp8idx.paged_block_attn_workspace(128) - 1)), INVALID, b"needed")
    for stride in ((512, 128, 2), (516, 128, 1), (512, 132, 1)):
        refused(lib, f(*attn_args(q=strided(_t(BF16, (5, 4, 128), 0x100000), *stride))), INVALID, b"rows must")
    for stride in ((512, 64, 1), (128, 128, 1), (0, 128, 1)):
        refused(lib, f(*attn_args(out=strided(_t(BF16, (5, 4, 128), 0x500000), *stride))), INVALID, b"rows overlap")
    assert f(*attn_args(T=0)) == fp8idx.FP8IDX_OK
    assert f(*attn_args(T=0, B=0, mb=0)) == fp8idx.FP8IDX_OK


def test_block_attention_overlaps(lib):
    f = lib.fp8_paged_block_attn
    size = 9 * 2 * (16 * 256 + 16)
    for at in (0x100000, 0x100010, 0x800000 + size - 16, 0x200000, 0x300000 - 16, 0x400000, 0x600000, 0x10000000):
        refused(lib, f(*attn_args(out=_t(BF16, (5, 4, 128), at))), INVALID, b"overlap")
    for at in (0x100000, 0x800000, 0x200000 + 4, 0x300004, 0x400000 - 4, 0x500000, 0x10000000 + 256):
        refused(lib, f(*attn_args(lse=_t(F32, (5, 4), at))), INVALID, b"overlap")
    for at in (0x100000, 0x800000, 0x500000):
        refused(lib, f(*attn_args(ws=at)), INVALID, b"overlap")


def test_binding_refuses_other_workspaces(monkeypatch):
    q = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    for ws in (torch.zeros(100, dtype=torch.float32), torch.zeros((100, 2), dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            fp8idx.fp8_paged_block_attn(q, q, q, q, q, 1.0, q, workspace=ws)


def test_binding_keeps_whole_numbers_whole(monkeypatch):
    """Numbers past 32 bits are refused, not cut to their lower bits."""
    x = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="window"):
        fp8idx.fp8_paged_block_attn(x, x, x, x, x, 1.0, x, window=5 - 2**32, workspace=torch.zeros(9, dtype=torch.uint8))
    monkeypatch.setattr(_native, "_descs", lambda *t: [None] * len(t))
    with pytest.raises(ValueError, match="rot_start"):
        fp8idx.head_norm_rope(x, None, x, x, x, rot_start=2**32)
    for sizes in ((2**32 + 64, 128), (64, 2**32 + 128)):
        with pytest.raises(ValueError, match="32 bits"):
            fp8idx.kv_block_page_bytes(*sizes)
    with pytest.raises(ValueError, match="head_dim"):
        fp8idx.paged_block_attn_workspace(2**32 + 128)


# --------------------------------------------------------------- definitions
def test_definition_of_the_rotation_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y, _ = ref.head_norm_rope(x, [1], [math.pi / 2], rot_start=2)  # elements 2 and 3: (3, 4) -> (-4, 3)
    assert np.allclose(y[0, 0], [1, 2, -4, 3, 5, 6, 7, 8])
    y, _ = ref.head_norm_rope(x, [2], [math.pi / 2, 0.0], rope_scale=2.0)  # (0, 2) by half a turn, (1, 3) by none
    assert np.allclose(y[0, 0], [-2, 4, -6, 8, 5, 6, 7, 8])
    y, _ = ref.head_norm_rope(x, [1], [0.0, math.pi / 2], interleaved=True)
    assert np.allclose(y[0, 0], [1, 2, -4, 3, 5, 6, 7, 8])
    y, _ = ref.head_norm_rope(np.full((1, 1, 4), 3.0), [5], [], "rms", weight=np.array([1, 2, 3, 4.0]), eps=0)
    assert np.allclose(y[0, 0], [1, 2, 3, 4])
    y, _ = ref.head_norm_rope(np.array([[[1.0, 3.0]]]), [5], [], "layer", bias=np.array([1, 1.0]), eps=0)
    assert np.allclose(y[0, 0], [0, 2])


def test_definition_of_block_scales_by_hand():
    bs, D = 16, 64
    cache = np.zeros((2, 1, ref.block_page_bytes(bs, D)), np.uint8)
    x = np.zeros((2, 1, D), np.float32)
    x[0, 0, :3], x[1, 0, 0] = [448, -7, 0.5], 1
    ref.store_blocks(cache, [16, 17], x, 2 * x, bs)

    def codes(t, part):
        return ref.e4m3_values()[cache[1, 0, (2 * t + part) * D: (2 * t + part) * D + 3]].tolist()

    def scales():
        return cache[1, 0, bs * 2 * D: bs * 2 * D + 8].copy().view(np.float32).tolist()
    assert scales() == [1, 2] and codes(0, 0) == codes(0, 1) == [448, -7, 0.5] and codes(1, 0) == [1, 0, 0]
    # a token that needs 2.5 times the keys' scale: twice doubled; the values' is enough
    ref.store_blocks(cache, [18], x[:1] * 2.5, x[:1], bs)
    assert scales() == [4, 2] and codes(0, 0) == [112, -1.75, 0.125] and codes(2, 0) == [288, -4.5, 0.3125]
    assert codes(0, 1) == [448, -7, 0.5] and codes(2, 1) == [224, -3.5, 0.25]
    assert not cache[0].any()
    # the block anew
    ref.store_blocks(cache, [16], x[:1] / 448, x[:1], bs)
    assert scales() == [np.float32(1) / np.float32(448), 1]
    assert ref.block_runs([3, 4, 15, 16, 17, -1, 18, 99], 64, 16) == [(0, 2), (2, 1), (3, 2), (6, 1)]


def test_definition_of_block_attention_by_hand():
    """Two tokens of equal score: the mean of their values, lse = s + ln 2; a
    window of one sees the last."""
    D, bs = 64, 16
    cache = np.zeros((1, 1, ref.block_page_bytes(bs, D)), np.uint8)
    k = np.ones((2, 1, D), np.float32)
    v = np.stack([np.full((1, D), 2.0), np.full((1, D), 4.0)]).astype(np.float32)
    ref.store_blocks(cache, [0, 1], k, v, bs)
    args = (cache, np.zeros((1, 1), int), [2], [0, 2], bs, 1.0)
    out, lse, *_ = ref.block_attention(np.full((3, 1, D), 0.5), *args)
    assert np.allclose(out[:2, 0, 0], [2, 3]) and np.allclose(lse[:2, 0], [32, 32 + np.log(2)]) and np.isnan(lse[2]).all()
    out, _, *_ = ref.block_attention(np.full((2, 1, D), 0.5), *args, window=1)
    assert np.allclose(out[:, 0, 0], [2, 4])
