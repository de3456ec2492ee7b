"""The operators in the order in which a serving step uses them, over a
prompt chunk and the decode steps after it: tables -> index keys, keys and
values into the caches -> logits -> top-k -> attention."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as ref
from oracle import topk as T
from parity import assert_rows_close
from serving import assert_attention, bf16

pytestmark = pytest.mark.gpu

INDEX_HEADS, HEADS, KV_HEADS, D = 32, 16, 2, 128


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    m.device_status()
    return m


class Server:
    """Caches, tables and free list of a few requests, on both sides."""

    def __init__(self, fp8idx, rng, batch, max_len, block_size):
        self.m, self.rng, self.bs, self.batch, self.max_len = fp8idx, rng, block_size, batch, max_len
        per = -(-max_len // block_size)
        blocks = batch * per + 3
        self.h = {"tables": np.full((batch, per), -1, np.int32),
                  "free": rng.permutation(blocks).astype(np.int32), "count": blocks,
                  "index": rng.integers(0, 256, (blocks, block_size * (D + 4)), dtype=np.uint8),
                  "kv": rng.integers(0, 256, (blocks, KV_HEADS, ref.page_bytes(block_size, D)), dtype=np.uint8)}
        # (the logits kernels read whole pages: every slot holds a key)
        ref.store_index(self.h["index"], np.arange(blocks * block_size),
                        rng.standard_normal((blocks * block_size, D)).astype(np.float32), block_size)
        self.d = {n: torch.from_numpy(np.array(x)).cuda() for n, x in self.h.items() if n != "count"}
        self.d["count"] = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        self.old = np.zeros(batch, np.int32)

    def inputs(self, new, k):
        """One step's inputs and output buffers on the GPU."""
        rng, rows = self.rng, int(new.sum())
        x = {"old": self.old.copy(), "new": new, "ik": bf16(rng.standard_normal((rows, D))),
             "k": bf16(rng.standard_normal((rows, KV_HEADS, D))), "v": bf16(rng.standard_normal((rows, KV_HEADS, D))),
             "iq": ref.quantise_rows(rng.standard_normal((rows, INDEX_HEADS, D)))[0],
             "w": rng.standard_normal((rows, INDEX_HEADS)).astype(np.float32),
             "q": bf16(rng.standard_normal((rows, HEADS, D)))}
        g = {n: torch.from_numpy(a).cuda() for n, a in x.items()}
        for n in ("ik", "k", "v", "q"):
            g[n] = g[n].to(torch.bfloat16)
        i32 = dict(dtype=torch.int32, device="cuda")
        g.update(ctx=torch.empty(self.batch, **i32), cu_new=torch.empty(self.batch + 1, **i32),
                 cu_seq=torch.empty(self.batch + 1, **i32), slots=torch.empty(rows, **i32), ks=torch.empty(rows, **i32),
                 ke=torch.empty(rows, **i32), counts=torch.empty(4, **i32), idx=torch.empty((rows, k), **i32),
                 out=torch.empty((rows, HEADS, D), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty((rows, HEADS), device="cuda"))
        return x, g

    def tables_and_store(self, g):
        d, m = self.d, self.m
        m.paged_step_tables(g["old"], g["new"], d["free"], d["count"], self.bs, d["tables"], g["ctx"], g["cu_new"],
                            g["slots"], g["counts"], cu_seq_lens=g["cu_seq"], cu_seqlen_ks=g["ks"], cu_seqlen_ke=g["ke"])
        m.fp8_paged_store(g["ik"], None, g["slots"], d["index"])
        m.fp8_paged_store(g["k"], g["v"], g["slots"], d["kv"])
        d["count"].copy_(g["counts"][2:3])

    def prompt(self, g, cols, k):
        self.tables_and_store(g)
        d, m = self.d, self.m
        g["logits"] = torch.empty((g["iq"].shape[0], cols), device="cuda")
        m.fp8_mqa_logits_paged(g["iq"], d["index"], d["tables"], g["cu_seq"], g["w"], g["ks"], g["ke"], g["logits"])
        m.fp8_mqa_topk(g["logits"], g["ks"], g["ke"], k, g["idx"])
        m.fp8_mqa_sparse_attn_paged(g["q"], d["kv"], d["tables"], g["cu_seq"], g["idx"], D**-0.5, g["out"], lse=g["lse"])

    def decode(self, g, n, k):
        self.tables_and_store(g)
        d, m, B = self.d, self.m, self.batch
        m.fp8_paged_mqa_logits(g["iq"].view(B, n, INDEX_HEADS, D), d["index"], g["w"], g["ctx"], d["tables"],
                               self.max_len, g["logits"])
        m.fp8_paged_topk(g["logits"], g["ctx"], n, self.max_len, k, g["idx"])
        m.fp8_paged_sparse_attn(g["q"].view(B, n, HEADS, D), d["kv"], g["idx"], d["tables"], D**-0.5,
                                g["out"].view(B, n, HEADS, D), lse=g["lse"])

    def check_state(self, x, g):
        """Tables and caches of the step, exactly; advances the host's state."""
        h = self.h
        want = ref.step_tables(x["old"], x["new"], h["free"], h["count"], self.bs, h["tables"], int(x["new"].sum()))
        for name, t in (("block_tables", self.d["tables"]), ("context_lens", g["ctx"]), ("cu_new_lens", g["cu_new"]),
                        ("cu_seq_lens", g["cu_seq"]), ("slot_mapping", g["slots"]), ("cu_seqlen_ks", g["ks"]),
                        ("cu_seqlen_ke", g["ke"]), ("counts", g["counts"])):
            assert np.array_equal(t.cpu().numpy(), want[name]), name
        h["tables"], h["count"] = want["block_tables"], int(want["counts"][2])
        ref.store_index(h["index"], want["slot_mapping"], x["ik"], self.bs)
        ref.store_kv(h["kv"], want["slot_mapping"], x["k"], x["v"], self.bs)
        assert np.array_equal(self.d["index"].cpu().numpy(), h["index"])
        assert np.array_equal(self.d["kv"].cpu().numpy(), h["kv"])
        self.old = want["context_lens"]
        return want

    def check_attention(self, x, g, **form):
        want = ref.sparse_attention(x["q"].astype(np.float64), self.h["kv"], g["idx"].cpu().numpy(), self.h["tables"],
                                    self.bs, D**-0.5, **form)
        assert_attention(g["out"].float().cpu().numpy(), g["lse"].cpu().numpy(), want)


@pytest.mark.parametrize("block_size", [1, 16, 64])
def test_prompt_then_decode(fp8idx, block_size):
    rng = np.random.default_rng(31 + block_size)
    orc = oracle.Oracle()
    B, n, k, max_len = 3, 2, 128, 512
    s = Server(fp8idx, rng, B, max_len, block_size)
    for new in (np.array([200, 1, 131], np.int32), np.array([40, 90, 5], np.int32)):  # two prompt chunks
        x, g = s.inputs(new, k)
        if block_size == 1:  # (the prompt's logits read pages of 16 tokens and more)
            s.tables_and_store(g)
            torch.cuda.synchronize()
            s.check_state(x, g)
            continue
        s.prompt(g, int(s.old.sum() + new.sum()), k)
        torch.cuda.synchronize()
        want = s.check_state(x, g)
        keys, scales = oracle.gather_paged_k(s.h["index"], s.h["tables"], want["cu_seq_lens"], block_size)
        logits = orc.mqa_logits(x["iq"], keys, scales, x["w"], want["cu_seqlen_ks"], want["cu_seqlen_ke"])
        got = g["logits"].cpu().numpy()
        assert_rows_close(got, logits)
        assert np.array_equal(g["idx"].cpu().numpy(),
                              T.topk_rows(got, *T.prefill_windows(want["cu_seqlen_ks"], want["cu_seqlen_ke"], got.shape[1]), k))
        s.check_attention(x, g, cu_seq_lens=want["cu_seq_lens"])
    for _ in range(3):  # decode steps, each also from a captured graph
        x, g = s.inputs(np.full(B, n, np.int32), k)
        g["logits"] = torch.full((B * n, max_len), float("-inf"), device="cuda")
        before = {name: t.clone() for name, t in s.d.items()}
        s.decode(g, n, k)
        torch.cuda.synchronize()
        eager = {name: g[name].clone() for name in ("out", "lse", "idx", "slots")}
        after = {name: t.clone() for name, t in s.d.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.decode(g, n, k)
        for name, t in before.items():
            s.d[name].copy_(t)
        for name in eager:
            g[name].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in eager.items():
            assert torch.equal(g[name], t), name
        for name, t in after.items():
            assert torch.equal(s.d[name], t), name
        want = s.check_state(x, g)
        logits = orc.paged_mqa_logits(x["iq"].reshape(B, n, INDEX_HEADS, D), s.h["index"], x["w"], want["context_lens"],
                                      np.maximum(s.h["tables"], 0), block_size, max_len)
        got = g["logits"].cpu().numpy()
        assert_rows_close(got, logits)
        assert np.array_equal(g["idx"].cpu().numpy(),
                              T.topk_rows(got, *T.decode_windows(want["context_lens"], n, max_len), k))
        s.check_attention(x, g, next_n=n)
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
