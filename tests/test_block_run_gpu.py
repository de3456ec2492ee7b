"""The operators of dense attention in the order in which a serving step uses
them, over prompt chunks, steps that mix them with decode rows, and captured
decode steps: tables -> norms and rotation -> the quantising store -> attention."""
import numpy as np
import pytest
import torch

from block_cases import assert_block_attention
from oracle import serving as ref
from test_block_store_gpu import same
from test_head_norm_rope_gpu import tolerance

pytestmark = pytest.mark.gpu

H, HK = 12, 3


@pytest.fixture(scope="module")
def fp8idx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_fp8_gb300 as m
    m.library()
    m.device_status()
    return m


class Server:
    """Cache, tables and free list of a few requests, on both sides."""

    def __init__(self, fp8idx, rng, batch, max_len, bs, D, window):
        self.m, self.rng, self.bs, self.D, self.batch, self.window = fp8idx, rng, bs, D, batch, window
        per = -(-max_len // bs)
        blocks = batch * per + 3
        self.tables, self.count = np.full((batch, per), -1, np.int32), blocks
        self.free = rng.permutation(blocks).astype(np.int32)
        self.cache = rng.integers(0, 256, (blocks, HK, ref.block_page_bytes(bs, D)), dtype=np.uint8)
        self.old = np.zeros(batch, np.int32)
        self.inv = torch.tensor([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float32)
        self.w = {n: (1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for n in "qk"}
        self.d = {n: torch.from_numpy(np.array(x)).cuda() for n, x in
                  (("tables", self.tables), ("free", self.free), ("cache", self.cache))}
        self.d.update(count=torch.tensor([blocks], dtype=torch.int32, device="cuda"), inv=self.inv.cuda(),
                      qw=torch.from_numpy(self.w["q"]).cuda(), kw=torch.from_numpy(self.w["k"]).cuda(),
                      ws=torch.empty(fp8idx.paged_block_attn_workspace(D), dtype=torch.uint8, device="cuda"))

    def inputs(self, new, pad=0):
        """One step's projections [rows, (H + 2 HK) D] and buffers."""
        rows = int(new.sum()) + pad
        i32 = dict(dtype=torch.int32, device="cuda")
        pos = np.full(rows, -1, np.int32)
        pos[: rows - pad] = np.concatenate([o + np.arange(n) for o, n in zip(self.old, new)])
        return {"old": torch.from_numpy(self.old.copy()).cuda(), "new": torch.from_numpy(new).cuda(),
                "qkv": torch.from_numpy(self.rng.standard_normal((rows, (H + 2 * HK) * self.D)).astype(np.float32)).to(
                    torch.bfloat16).cuda(), "pos": torch.from_numpy(pos).cuda(),
                "ctx": torch.empty(self.batch, **i32), "cu": torch.empty(self.batch + 1, **i32),
                "slots": torch.empty(rows, **i32), "counts": torch.empty(4, **i32),
                "out": torch.full((rows, H, self.D), float("nan"), dtype=torch.bfloat16, device="cuda"),
                "lse": torch.full((rows, H), float("nan"), device="cuda")}

    def parts(self, g):
        rows, D = g["qkv"].shape[0], self.D
        x = g["qkv"].view(rows, H + 2 * HK, D)
        return x[:, :H], x[:, H: H + HK], x[:, H + HK:]

    def step(self, g):
        d, m = self.d, self.m
        q, k, v = self.parts(g)
        m.paged_step_tables(g["old"], g["new"], d["free"], d["count"], self.bs, d["tables"], g["ctx"], g["cu"], g["slots"],
                            g["counts"])
        m.head_norm_rope(q, k, g["pos"], d["inv"], q, k, norm="rms", q_weight=d["qw"], k_weight=d["kw"])
        m.fp8_paged_block_store(k, v, g["slots"], d["cache"])
        m.fp8_paged_block_attn(q, d["cache"], d["tables"], g["ctx"], g["cu"], self.D**-0.5, g["out"], lse=g["lse"],
                               window=self.window, workspace=d["ws"])
        d["count"].copy_(g["counts"][2:3])

    def check(self, g, before):
        """before: the projections as they were."""
        rows, D = before.shape[0], self.D
        pos = g["pos"].cpu().numpy()
        want = ref.step_tables(g["old"].cpu().numpy(), g["new"].cpu().numpy(), self.free, self.count, self.bs, self.tables, rows)
        for name, t in (("block_tables", self.d["tables"]), ("context_lens", g["ctx"]), ("cu_new_lens", g["cu"]),
                        ("slot_mapping", g["slots"]), ("counts", g["counts"])):
            assert np.array_equal(t.cpu().numpy(), want[name]), name
        self.tables, self.count, self.old = want["block_tables"], int(want["counts"][2]), want["context_lens"]
        x = before.double().cpu().numpy().reshape(rows, H + 2 * HK, D)
        q, k, v = (t.double().cpu().numpy() for t in self.parts(g))
        assert np.array_equal(v, x[:, H + HK:])
        live = pos >= 0
        for got, a, w in ((q, x[:, :H], self.w["q"]), (k, x[:, H: H + HK], self.w["k"])):
            y, terms = ref.head_norm_rope(a, pos, self.inv.double().numpy(), "rms", w)
            assert (np.abs(got - y) <= tolerance(a, terms, y, torch.bfloat16, "rms"))[live].all()
            assert np.array_equal(got[~live], a[~live])
        ref.store_blocks(self.cache, want["slot_mapping"], k.astype(np.float32), v.astype(np.float32), self.bs)
        got = self.d["cache"].cpu().numpy()
        same(got, self.cache, self.bs, D)
        self.cache = got  # (0 and -0 as they are)
        figures = ref.block_attention(q, self.cache, self.tables, want["context_lens"], want["cu_new_lens"], self.bs, D**-0.5,
                                      self.window)
        assert_block_attention(g["out"].float().cpu().numpy(), g["lse"].cpu().numpy(), figures)


@pytest.mark.parametrize("bs,D,window", [(16, 128, 0), (64, 64, 0), (32, 128, 70), (128, 64, 200)])
def test_prompts_then_decode(fp8idx, bs, D, window):
    rng = np.random.default_rng(bs + D)
    s = Server(fp8idx, rng, 4, 700, bs, D, window)
    for new in ([200, 1, 131, 0], [40, 90, 5, 260], [1, 1, 150, 1]):  # prompt chunks, decode rows among them
        g = s.inputs(np.array(new, np.int32), pad=7)
        before = g["qkv"].clone()
        s.step(g)
        torch.cuda.synchronize()
        s.check(g, before)
    for n in (1, 1, 3):  # decode steps, each also from a captured graph
        g = s.inputs(np.full(4, n, np.int32))
        before, state = g["qkv"].clone(), {name: t.clone() for name, t in s.d.items() if name != "ws"}
        s.step(g)
        torch.cuda.synchronize()
        eager = {name: g[name].clone() for name in ("out", "lse", "slots", "qkv")}
        after = {name: s.d[name].clone() for name in state}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step(g)
        for name, t in state.items():
            s.d[name].copy_(t)
        g["qkv"].copy_(before)
        g["out"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for name, t in eager.items():
            assert torch.equal(g[name], t), name
        for name, t in after.items():
            assert torch.equal(s.d[name], t), name
        s.check(g, before)
    assert fp8idx.device_status() == fp8idx.FP8IDX_OK
