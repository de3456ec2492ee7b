"""Refusals of the operators around the indexer (CPU: host checks with fake
pointers that are never dereferenced, before any CUDA call), and their plain
definitions on hand cases."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_attention_fp8_gb300 as fp8idx
from oracle import serving as ref
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


def test_page_bytes(lib):
    for bs in (1, 16, 32, 64, 128):
        for d in (64, 128):
            assert fp8idx.kv_page_bytes(bs, d) == ref.page_bytes(bs, d)
    assert fp8idx.kv_page_bytes(8, 128) == 0 and fp8idx.kv_page_bytes(64, 96) == 0


def step_args(B=3, T=10, mb=4, **kw):
    at = iter(range(0x100000, 0x200000, 0x1000))
    a = dict(old=_t(I32, (B,), next(at)), new=_t(I32, (B,), next(at)), free=_t(I32, (9,), next(at)),
             count=_t(I32, (1,), next(at)), bs=16, bt=_t(I32, (B, mb), next(at)), ctx=_t(I32, (B,), next(at)),
             cu=_t(I32, (B + 1,), next(at)), slots=_t(I32, (T,), next(at)), counts=_t(I32, (4,), next(at)),
             seq=_t(I32, (B + 1,), next(at)), ks=_t(I32, (T,), next(at)), ke=_t(I32, (T,), next(at)))
    a.update(kw)
    return [R(v) if isinstance(v, ctypes.Structure) else v for v in a.values()] + [None]


def test_step_tables_refusals(lib):
    f = lib.fp8idx_paged_step_tables
    refused(lib, f(*step_args(old=None)), INVALID, b"old_lens")
    refused(lib, f(*step_args(new=_t(I32, (4,)))), INVALID, b"new_lens")
    refused(lib, f(*step_args(count=_t(I32, (2,)))), INVALID, b"free_count")
    refused(lib, f(*step_args(counts=_t(I32, (3,)))), INVALID, b"counts")
    refused(lib, f(*step_args(slots=_t(F32, (10,)))), INVALID, b"slot_mapping")
    refused(lib, f(*step_args(ks=_t(I32, (9,)))), INVALID, b"cu_seqlen_ks")
    refused(lib, f(*step_args(bt=_t(I32, (2, 4)))), INVALID, b"block_tables")
    refused(lib, f(*step_args(bs=8)), UNSUPPORTED, b"block_size")
    refused(lib, f(*step_args(bs=0)), UNSUPPORTED, b"block_size")
    refused(lib, f(*step_args(B=4097)), UNSUPPORTED, b"batch")
    refused(lib, f(*step_args(mb=1 << 27)), UNSUPPORTED, b"2^31")
    refused(lib, f(*step_args(ctx=_t(I32, (3,), 0x100000))), INVALID, b"overlaps an input")   # old_lens in place
    refused(lib, f(*step_args(ctx=_t(I32, (3,), 0x107008))), INVALID, b"two outputs")
    strided = _t(I32, (3,), 0x300000)
    strided.stride[0] = 2
    refused(lib, f(*step_args(old=strided)), INVALID, b"old_lens")


def test_store_refusals(lib):
    f = lib.fp8_paged_store
    k, slots, kv = _t(BF16, (5, 2, 128)), _t(I32, (5,)), _t(U8, (4, 2, 16 * 264))
    refused(lib, f(None, R(k), R(slots), R(kv), None), INVALID, b"k: null")
    refused(lib, f(R(_t(I32, (5, 2, 128))), R(k), R(slots), R(kv), None), INVALID, b"dtype")
    refused(lib, f(R(k), R(_t(F16, (5, 2, 128))), R(slots), R(kv), None), INVALID, b"v: wrong dtype")
    refused(lib, f(R(k), R(_t(BF16, (5, 1, 128))), R(slots), R(kv), None), INVALID, b"shape of k")
    refused(lib, f(R(k), R(k), R(_t(I32, (4,))), R(kv), None), INVALID, b"slot_mapping")
    refused(lib, f(R(k), R(k), R(slots), R(_t(U8, (4, 2, 16 * 264 + 16))), None), INVALID, b"page")
    refused(lib, f(R(k), R(k), R(slots), R(_t(U8, (4, 2, 8 * 264))), None), UNSUPPORTED, b"block_size")
    refused(lib, f(R(k), R(k), R(slots), R(_t(U8, (4, 3, 16 * 264))), None), INVALID, b"heads")
    refused(lib, f(R(k), R(k), R(slots), R(_t(U8, (4, 2, 16 * 264), 0x1008)), None), INVALID, b"aligned")
    refused(lib, f(R(_t(BF16, (5, 2, 128), 0x1008)), R(k), R(slots), R(kv), None), INVALID, b"aligned")
    odd = _t(BF16, (5, 2, 128))
    odd.stride[0] = 260
    refused(lib, f(R(odd), R(k), R(slots), R(kv), None), INVALID, b"aligned")
    odd = _t(BF16, (5, 2, 128))
    odd.stride[2] = 2
    refused(lib, f(R(odd), R(k), R(slots), R(kv), None), INVALID, b"inner stride")
    over = _t(U8, (4, 2, 16 * 264))
    over.stride[0] = over.stride[1] = 16 * 264
    refused(lib, f(R(k), R(k), R(slots), R(over), None), INVALID, b"overlap")
    refused(lib, f(R(k), R(k), R(slots), R(_t(U8, (1 << 27, 2, 16 * 264))), None), UNSUPPORTED, b"2^31")
    k96 = _t(BF16, (5, 2, 96))
    refused(lib, f(R(k96), R(k96), R(slots), R(_t(U8, (4, 2, 16 * 200))), None), UNSUPPORTED, b"head_dim")
    # the index cache
    k2 = _t(F32, (5, 128))
    refused(lib, f(R(k2), None, R(slots), R(_t(U8, (4, 100))), None), INVALID, b"head_dim+4")
    refused(lib, f(R(k2), None, R(slots), R(_t(U8, (4, 5 * 132))), None), UNSUPPORTED, b"block_size")
    refused(lib, f(R(k), None, R(slots), R(_t(U8, (4, 64 * 132))), None), INVALID, b"ndim")
    refused(lib, f(R(k2), None, R(slots), R(kv), None), INVALID, b"ndim")


def attn_args(q=None, kv=None, idx=None, bt=None, scale=1.0, out=None, lse=None, opts=None):
    q = q or _t(BF16, (2, 3, 8, 128))
    return [R(q), R(kv or _t(U8, (9, 2, 16 * 264))), R(idx or _t(I32, (6, 50))), R(bt or _t(I32, (2, 5))), scale,
            R(out or _t(BF16, tuple(q.shape[:q.ndim]))), None if lse is None else R(lse),
            None if opts is None else R(opts._c()), None]


def test_decode_attention_refusals(lib):
    f = lib.fp8_paged_sparse_attn
    refused(lib, f(*attn_args(q=_t(F32, (2, 3, 8, 128)))), INVALID, b"q: wrong dtype")
    refused(lib, f(*attn_args(q=_t(BF16, (6, 8, 128)))), INVALID, b"ndim")
    refused(lib, f(*attn_args(q=_t(BF16, (2, 3, 8, 96)))), UNSUPPORTED, b"head_dim")
    # (a page of 4224 bytes is that of 31 tokens of 64 values: 31 * 136 = 4216, padded)
    refused(lib, f(*attn_args(q=_t(BF16, (2, 3, 8, 64)))), UNSUPPORTED, b"block_size 31")
    refused(lib, f(*attn_args(kv=_t(U8, (9, 2, 16 * 264 + 32)))), INVALID, b"page")
    refused(lib, f(*attn_args(out=_t(BF16, (2, 3, 4, 128)))), INVALID, b"shape of q")
    refused(lib, f(*attn_args(q=_t(BF16, (2, 3, 7, 128)))), INVALID, b"multiple")
    refused(lib, f(*attn_args(q=_t(BF16, (2, 3, 258, 128)))), UNSUPPORTED, b"heads per key head")
    refused(lib, f(*attn_args(idx=_t(I32, (5, 50)))), INVALID, b"indices")
    refused(lib, f(*attn_args(idx=_t(I32, (6, 2049)))), UNSUPPORTED, b"k=2049")
    refused(lib, f(*attn_args(idx=_t(I32, (6, 0)))), UNSUPPORTED, b"k=0")
    refused(lib, f(*attn_args(bt=_t(I32, (3, 5)))), INVALID, b"block_tables")
    refused(lib, f(*attn_args(bt=_t(I32, (2, 0)))), INVALID, b"block table")
    refused(lib, f(*attn_args(lse=_t(F32, (6, 7)))), INVALID, b"lse")
    refused(lib, f(*attn_args(scale=float("inf"))), INVALID, b"softmax_scale")
    refused(lib, f(*attn_args(scale=float("nan"))), INVALID, b"softmax_scale")
    refused(lib, f(*attn_args(opts=fp8idx.Options(num_ctas=3))), UNSUPPORTED, b"num_ctas")
    refused(lib, f(*attn_args(q=_t(BF16, (2, 3, 8, 128), 0x1002))), INVALID, b"aligned")
    odd = _t(BF16, (2, 3, 8, 128))
    odd.stride[1] = 8 * 128 + 4
    refused(lib, f(*attn_args(q=odd)), INVALID, b"aligned")
    refused(lib, f(*attn_args(scale=3e38)), INVALID, b"softmax_scale")
    for dim in range(3):
        same = _t(BF16, (2, 3, 8, 128))
        same.stride[dim] = 0
        refused(lib, f(*attn_args(out=same)), INVALID, b"overlap")
    back = _t(I32, (6, 50))
    back.stride[0] = -50
    refused(lib, f(*attn_args(idx=back)), INVALID, b"indices")


def test_prefill_attention_refusals(lib):
    f = lib.fp8_mqa_sparse_attn_paged
    q, kv, idx, out = _t(BF16, (6, 8, 128)), _t(U8, (9, 2, 16 * 264)), _t(I32, (6, 50)), _t(BF16, (6, 8, 128))
    bt, cu = _t(I32, (2, 5)), _t(I32, (3,))
    refused(lib, f(R(q), R(kv), R(bt), R(_t(I32, (2,))), R(idx), 1.0, R(out), None, None, None), INVALID, b"cu_seq_lens")
    refused(lib, f(R(q), R(kv), R(bt), None, R(idx), 1.0, R(out), None, None, None), INVALID, b"cu_seq_lens")
    refused(lib, f(R(q), R(kv), R(_t(I32, (4097, 5))), R(_t(I32, (4098,))), R(idx), 1.0, R(out), None, None, None),
            UNSUPPORTED, b"requests")
    refused(lib, f(R(q), R(kv), R(_t(I32, (0, 5))), R(cu), R(idx), 1.0, R(out), None, None, None), INVALID, b"block table")


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        fp8idx.fp8_paged_store(torch.zeros(2, 128), None, torch.zeros(2, dtype=torch.int32),
                               torch.zeros(2, 132, dtype=torch.uint8))


class OnDevice:
    """A host tensor that says it lies on a device."""

    def __init__(self, t, at):
        self.t, self.at = t, at

    def get_device(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_descriptors_and_devices(monkeypatch):
    from sparse_attention_fp8_gb300 import _native
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for t in (torch.zeros(5, dtype=torch.int32), torch.zeros(10)[::2], torch.zeros((3, 4), dtype=torch.uint8).t(),
              torch.zeros((2, 3, 4, 5)), torch.zeros((0, 7)), torch.zeros(()), torch.zeros((2, 3, 4))):
        assert _native._descs(OnDevice(t, 1), None) == [_native._pack(t, t.data_ptr()), None], t.shape
    with pytest.raises(TypeError):
        _native._descs(OnDevice(torch.zeros(3, dtype=torch.int64), 1))
    with pytest.raises(ValueError):
        _native._descs(OnDevice(torch.zeros((1, 1, 1, 1, 1)), 1))
    one, other = OnDevice(torch.zeros(3), 1), OnDevice(torch.zeros(3), 0)
    for ts in ((other,), (one, other), (one, torch.zeros(3))):
        with pytest.raises(ValueError):
            _native._descs(*ts)


def test_definition_step_tables_by_hand():
    tables = np.array([[7, -1, -1], [3, 4, -1]], np.int32)
    got = ref.step_tables([2, 8], [3, 1], np.array([20, 21, 22, 23]), 4, 4, tables, 6)
    # request 0: positions 2, 3 in block 7, position 4 in the first block dealt; request 1: position 8
    assert got["slot_mapping"].tolist() == [30, 31, 92, 88, -1, -1]
    assert got["block_tables"].tolist() == [[7, 23, -1], [3, 4, 22]]
    assert got["context_lens"].tolist() == [5, 9] and got["cu_seq_lens"].tolist() == [0, 5, 14]
    assert got["cu_seqlen_ks"].tolist() == [0, 0, 0, 5, 0, 0] and got["cu_seqlen_ke"].tolist() == [3, 4, 5, 14, 0, 0]
    assert got["counts"].tolist() == [4, 2, 2, 0] and got["cu_new_lens"].tolist() == [0, 3, 4]


def test_definition_of_codes():
    """The code table against torch's float8 type, and a row by hand."""
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(ref.e4m3_values(), nan=-1), np.nan_to_num(want, nan=-1))
    codes, scale = ref.quantise_rows(np.array([[0.0, 448.0, -224.0, 1.0625], [0.0] * 4]))
    assert scale.tolist() == [1.0, 0.0] and codes.tolist() == [[0, 0x7E, 0xF6, 0x38], [0, 0, 0, 0]]


def test_definition_of_attention_by_hand():
    """Two tokens of equal score: the mean of their values, lse = s + ln 2."""
    D, bs = 64, 16
    cache = np.zeros((1, 1, ref.page_bytes(bs, D)), np.uint8)
    k = np.ones((2, 1, D), np.float32)
    v = np.stack([np.full((1, D), 2.0), np.full((1, D), 4.0)]).astype(np.float32)
    ref.store_kv(cache, [3, 9], k, v, bs)
    out, lse, *_ = ref.sparse_attention(np.full((1, 1, D), 0.5), cache, np.array([[3, 9, -1]]), np.zeros((1, 1), int), bs,
                                        1.0, next_n=1)
    assert np.allclose(out, 3.0) and np.allclose(lse, 32 + np.log(2))


def strided(t, *stride):
    for i, s in enumerate(stride):
        t.stride[i] = s
    return t


@pytest.mark.parametrize("stride", [(128, 128, 128, 1), (8192, 128, 128, 1), (128, 256, 640, 1), (1024, 1024, 128, 1),
                                    (1024, 1920, 128, 1), (3 * 8 * 128 - 8, 8 * 128, 128, 1), (3 * 8 * 128, 8 * 128, 120, 1)])
def test_outputs_whose_rows_overlap(lib, stride):
    """Strides that are each no less than a row, but not next to one another."""
    out = strided(_t(BF16, (2, 3, 8, 128), 0x900000), *stride)
    refused(lib, lib.fp8_paged_sparse_attn(*attn_args(out=out)), INVALID, b"out: rows overlap")


def test_outputs_that_overlap_inputs(lib):
    f, g = lib.fp8_paged_sparse_attn, lib.fp8_mqa_sparse_attn_paged
    far = dict(q=_t(BF16, (2, 3, 8, 128), 0x10000), kv=_t(U8, (9, 2, 16 * 264), 0x100000), idx=_t(I32, (6, 50), 0x20000),
               bt=_t(I32, (2, 5), 0x30000), out=_t(BF16, (2, 3, 8, 128), 0x40000), lse=_t(F32, (6, 8), 0x50000))

    def moved(name, at):
        t = {"out": _t(BF16, (2, 3, 8, 128), at), "lse": _t(F32, (6, 8), at)}[name]
        refused(lib, f(*attn_args(**{**far, name: t})), INVALID, b"overlap")
    for at in (0x10000, 0x10000 + 12286, 0x10000 - 12286, 0x100010, 0x20004, 0x30008, 0x50000):
        moved("out", at)
    for at in (0x10000, 0x100000 + 9 * 2 * 16 * 264 - 4, 0x20000, 0x30000 - 4, 0x40000):
        moved("lse", at)
    # a head of every row of out lies on one of q's
    q = strided(_t(BF16, (2, 3, 8, 128), 0x10000), 3 * 8 * 1024, 8 * 1024, 1024)
    out = strided(_t(BF16, (2, 3, 8, 128), 0x10000 + 2 * (1024 - 120)), 3 * 8 * 1024, 8 * 1024, 1024)
    refused(lib, f(*attn_args(**{**far, "q": q, "out": out, "kv": _t(U8, (9, 2, 16 * 264), 0x1000000)})), INVALID, b"overlap")
    cu = _t(I32, (3,), 0x60000)
    refused(lib, g(R(_t(BF16, (6, 8, 128), 0x10000)), R(far["kv"]), R(far["bt"]), R(cu), R(far["idx"]), 1.0,
                   R(_t(BF16, (6, 8, 128), 0x60000 + 8)), None, None, None), INVALID, b"overlap")


def test_caches_that_overlap_rows(lib):
    f = lib.fp8_paged_store
    k, v, slots = _t(BF16, (5, 2, 128), 0x10000), _t(BF16, (5, 2, 128), 0x20000), _t(I32, (5,), 0x30000)
    size = 4 * 2 * 16 * 264
    for at in (0x10000, 0x20000 - size + 16, 0x30000):
        refused(lib, f(R(k), R(v), R(slots), R(_t(U8, (4, 2, 16 * 264), at)), None), INVALID, b"overlap")
    refused(lib, f(R(_t(F32, (5, 128), 0x10000)), None, R(slots), R(_t(U8, (4, 64 * 132), 0x10000 + 256)), None), INVALID,
            b"overlap")


def test_data_between_elements(lib):
    """A pointer that is no multiple of its element's size cannot be read or
    written by a kernel."""
    f = lib.fp8_paged_sparse_attn
    far = dict(q=_t(BF16, (2, 3, 8, 128), 0x10000), kv=_t(U8, (9, 2, 16 * 264), 0x100000), idx=_t(I32, (6, 50), 0x20000),
               bt=_t(I32, (2, 5), 0x30000), out=_t(BF16, (2, 3, 8, 128), 0x40000), lse=_t(F32, (6, 8), 0x50000))
    for name, by in (("out", 1), ("idx", 2), ("bt", 1), ("lse", 2)):
        t = _native_copy(far[name])
        t.data += by
        refused(lib, f(*attn_args(**{**far, name: t})), INVALID, b"aligned")
    refused(lib, lib.fp8idx_paged_step_tables(*step_args(counts=_t(I32, (4,), 0x300002))), INVALID, b"aligned")
    k, kv = _t(BF16, (5, 2, 128), 0x10000), _t(U8, (4, 2, 16 * 264), 0x100000)
    refused(lib, lib.fp8_paged_store(R(k), R(k), R(_t(I32, (5,), 0x20001)), R(kv), None), INVALID, b"aligned")
    # the calls that were there before
    refused(lib, lib.fp8_paged_topk(R(_t(F32, (6, 100), 0x10002)), R(_t(I32, (2,), 0x20000)), 3, 100, 10,
                                    R(_t(I32, (6, 10), 0x30000)), None), INVALID, b"aligned")


def _native_copy(t):
    c = type(t)()
    ctypes.memmove(R(c), R(t), ctypes.sizeof(t))
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_binding_of_the_logits_calls_refuses_16_bit_types(monkeypatch, dtype):
    """The types that the operators around them take: a TypeError of the
    binding, before the library is called, as for any other type."""
    from sparse_attention_fp8_gb300 import _native
    t = torch.zeros((2, 3, 4), dtype=dtype)
    with pytest.raises(TypeError, match="unsupported dtype"):
        _native._pack(t, t.data_ptr())
    monkeypatch.setattr(_native, "_desc", lambda x, out=False: _native._pack(x, x.data_ptr()))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fp8idx.fp8_paged_topk(t[0], i, 1, 4, 2, i, stream=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert len(_native._descs(OnDevice(t, 1))) == 1


def test_attention_of_no_rows(lib):
    """No rows, and no requests that they could belong to: nothing to do."""
    kv = _t(U8, (9, 2, 16 * 264), 0x100000)
    for reqs, blocks in ((2, 5), (0, 5), (0, 0)):
        assert lib.fp8_mqa_sparse_attn_paged(
            R(_t(BF16, (0, 8, 128))), R(kv), R(_t(I32, (reqs, blocks))), R(_t(I32, (reqs + 1,))), R(_t(I32, (0, 50))), 1.0,
            R(_t(BF16, (0, 8, 128))), R(_t(F32, (0, 8))), None, None) == fp8idx.FP8IDX_OK, lib.fp8idx_last_error()
    for blocks in (5, 0):
        assert lib.fp8_paged_sparse_attn(*attn_args(q=_t(BF16, (0, 3, 8, 128)), kv=kv, idx=_t(I32, (0, 50)),
                                                    bt=_t(I32, (0, blocks)))) == fp8idx.FP8IDX_OK, lib.fp8idx_last_error()
