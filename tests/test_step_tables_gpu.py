"""fp8idx_paged_step_tables on the GPU against the plain definition."""
import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    return m


def call(fp8idx, old, new, free, count, bs, tables, rows, prefill=True, stream=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    B = len(old)
    full = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    bt = d(tables)
    o = {"context_lens": full(B), "cu_new_lens": full(B + 1), "slot_mapping": full(rows), "counts": full(4)}
    x = {"cu_seq_lens": full(B + 1), "cu_seqlen_ks": full(rows), "cu_seqlen_ke": full(rows)} if prefill else {}
    args = (d(old), d(new), d(free), d([count]), bs, bt, *o.values())
    torch.cuda.synchronize()
    fp8idx.paged_step_tables(*args, **x, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in {"block_tables": bt, **o, **x}.items()}


def check(fp8idx, old, new, free, count, bs, tables, rows, **kw):
    got = call(fp8idx, old, new, free, count, bs, tables, rows, **kw)
    want = ref.step_tables(old, new, free, count, bs, tables, rows)
    for k in got:
        assert np.array_equal(got[k], want[k]), (k, got[k][:20], want[k][:20])
    return got


def batch(rng, B, bs, max_blocks, new_max, slack=8):
    new = rng.integers(0, new_max + 1, B)
    old = rng.integers(0, max(1, max_blocks * bs - new_max + 1), B)
    held = -(-old // bs)
    pool = rng.permutation(int(held.sum()) + int((-(-(old + new) // bs) - held).sum()) + slack).astype(np.int32)
    tables = np.full((B, max_blocks), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, : held[b]] = pool[at: at + held[b]]
        at += held[b]
    return old, new, pool[at:], tables


@pytest.mark.parametrize("bs", [1, 16, 32, 64, 128])
@pytest.mark.parametrize("B,new_max", [(1, 1), (3, 200), (33, 7), (257, 40)])
def test_matches_definition(fp8idx, B, new_max, bs):
    rng = np.random.default_rng(B * 1000 + bs)
    old, new, free, tables = batch(rng, B, bs, -(-600 // bs), new_max)
    check(fp8idx, old, new, free, len(free), bs, tables, int(new.sum()) + 13)
    check(fp8idx, old, new, free, len(free), bs, tables, int(new.sum()), prefill=False)


def test_largest_batch(fp8idx):
    rng = np.random.default_rng(9)
    old, new, free, tables = batch(rng, 4096, 16, 20, 9)
    check(fp8idx, old, new, free, len(free), 16, tables, int(new.sum()) + 1000)


def test_free_blocks_run_out(fp8idx):
    rng = np.random.default_rng(4)
    old, new, free, tables = batch(rng, 12, 16, 30, 100)
    for count in (0, 1, 17, len(free)):
        got = check(fp8idx, old, new, free, count, 16, tables, int(new.sum()))
        assert got["counts"][1] + got["counts"][2] == count
    # a count above the list, or below zero, is clamped
    check(fp8idx, old, new, free, len(free) + 50, 16, tables, int(new.sum()))
    check(fp8idx, old, new, free, -5, 16, tables, int(new.sum()))
    check(fp8idx, old, new, free[:0], 3, 16, tables, int(new.sum()))


def test_lengths_past_the_table_and_negative(fp8idx):
    tables = np.arange(12, dtype=np.int32).reshape(3, 4)
    free = np.arange(100, 120, dtype=np.int32)
    check(fp8idx, np.array([60, 64, 90]), np.array([10, 3, 5]), free, 20, 16, tables, 18)
    check(fp8idx, np.array([-3, 5, 0]), np.array([4, -9, 0]), free, 20, 16, tables, 9)
    big = 2**31 - 1
    check(fp8idx, np.array([big, 5, big]), np.array([big, 2, big]), free, 20, 16, tables, 40)


def test_fewer_rows_than_tokens_and_none(fp8idx):
    rng = np.random.default_rng(5)
    old, new, free, tables = batch(rng, 6, 32, 10, 50)
    check(fp8idx, old, new, free, len(free), 32, tables, 3)
    check(fp8idx, old, new, free, len(free), 32, tables, 0)
    check(fp8idx, old, new * 0, free, len(free), 32, tables, 5)
    empty = np.zeros(0, np.int64)
    check(fp8idx, empty, empty, free, len(free), 32, np.zeros((0, 4), np.int32), 7)


def test_block_ids_whose_slots_pass_31_bits(fp8idx):
    """A token whose slot does not fit in 32 bits gets slot -1."""
    tables = np.full((1, 4), -1, np.int32)
    free = np.array([7, 2**31 // 64, 2**31 // 64 - 1], np.int32)  # dealt from the end
    check(fp8idx, np.array([0]), np.array([192]), free, 3, 64, tables, 192)


def test_repeatable_captured_and_on_a_stream(fp8idx):
    rng = np.random.default_rng(6)
    old, new, free, tables = batch(rng, 40, 16, 30, 20)
    rows = int(new.sum()) + 5
    want = ref.step_tables(old, new, free, len(free), 16, tables, rows)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    bt = d(tables)
    ins = (d(old), d(new), d(free), d([len(free)]))
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (40, 41, rows, 4, 41, rows, rows)]
    kw = dict(cu_seq_lens=outs[4], cu_seqlen_ks=outs[5], cu_seqlen_ke=outs[6])
    fp8idx.paged_step_tables(*ins, 16, bt, *outs[:4], **kw)  # (loads the kernel before the capture)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8idx.paged_step_tables(*ins, 16, bt, *outs[:4], **kw)
    old2, new2, free2, tables2 = batch(rng, 40, 16, 30, 3)
    for (o, n, f, tb) in ((old, new, free, tables), (old2, new2, free2, tables2)):
        m = min(len(f), len(free))
        ins[0].copy_(d(o)), ins[1].copy_(d(n)), bt.copy_(d(tb)), ins[2][:m].copy_(d(f[:m])), ins[3].fill_(m)
        for t in outs:
            t.fill_(-5)
        g.replay()
        g.replay()  # a second call on the same state changes nothing
        torch.cuda.synchronize()
        w = ref.step_tables(o, n, np.concatenate([f[:m], free[m:]]) if m < len(free) else f, m, 16, tb, rows)
        for k, t in zip(("context_lens", "cu_new_lens", "slot_mapping", "counts", "cu_seq_lens", "cu_seqlen_ks",
                         "cu_seqlen_ke"), outs):
            assert np.array_equal(t.cpu().numpy(), w[k]), k
        assert np.array_equal(bt.cpu().numpy(), w["block_tables"])
    assert want["counts"][0] == new.sum()


def test_strided_tables(fp8idx):
    """A block table that is a slice of a wider one: the rest stays."""
    rng = np.random.default_rng(8)
    old, new, free, tables = batch(rng, 5, 16, 12, 30)
    wide = torch.full((5, 40), 4242, dtype=torch.int32, device="cuda")
    view = wide[:, 9:21]
    view.copy_(torch.from_numpy(tables))
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    rows = int(new.sum())
    o = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (5, 6, rows, 4)]
    fp8idx.paged_step_tables(d(old), d(new), d(free), d([len(free)]), 16, view, *o)
    want = ref.step_tables(old, new, free, len(free), 16, tables, rows)
    assert np.array_equal(view.cpu().numpy(), want["block_tables"])
    assert (wide[:, :9] == 4242).all() and (wide[:, 21:] == 4242).all()


def test_outputs_between_the_rows_of_a_table(fp8idx):
    """The block table as columns of a wider tensor whose other columns hold
    a step's vectors: nothing overlaps."""
    rng = np.random.default_rng(10)
    old, new, free, tables = batch(rng, 5, 16, 12, 30)
    wide = torch.full((5, 60), 4242, dtype=torch.int32, device="cuda")
    view, ctx, cu, count, counts = wide[:, 9:21], wide[0, 30:35], wide[1, 30:36], wide[2, 30:31], wide[3, 30:34]
    view.copy_(torch.from_numpy(tables))
    count.fill_(len(free))
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    rows = int(new.sum())
    slots = torch.empty(rows, dtype=torch.int32, device="cuda")
    fp8idx.paged_step_tables(d(old), d(new), d(free), count, 16, view, ctx, cu, slots, counts)
    want = ref.step_tables(old, new, free, len(free), 16, tables, rows)
    for t, name in ((view, "block_tables"), (ctx, "context_lens"), (cu, "cu_new_lens"), (counts, "counts"),
                    (slots, "slot_mapping")):
        assert np.array_equal(t.cpu().numpy(), want[name]), name
    assert (wide[:, :9] == 4242).all() and (wide[:, 21:30] == 4242).all() and (wide[:, 36:] == 4242).all()
