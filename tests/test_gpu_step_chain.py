"""A serving step of requests that share a prompt, as a program runs it: pages and slots for the new
rows, head norms and rotary positions, the rows stored at their slots, decode attention with the
prompt read once.  Eagerly and replayed from a graph, against a model of the step in 64 bits that
keeps each request's rows by itself.

Bars: k as stored is rounded once to bf16 (2^-8 of itself) from values good to 2^-18 of a pair's
length, so the model takes the rows as the library stored them and is compared with them by that
bar; the attention over equal rows then has the bars of tests/test_gpu_shared.py: 2^-8 of
|o| + sum a |v| over the shared rows, 2^-12 max |v|, lse 1e-4."""
import math

import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa
from kv_cache_serving_gb300 import workloads as wl
from kv_cache_serving_gb300.session import DecodeBatch, PagePool

pytestmark = pytest.mark.gpu
BF, U = torch.bfloat16, 2.0 ** -8


class Step:
    """Twelve requests in three groups of one prompt each, their fused projection and pool."""

    def __init__(self, masked, seed=7):
        cfg = wl.scaled(wl.WORKLOADS["mixed-serving"], batch=12, hq=8, hkv=2, prompt=(40, 90),
                        seq=("after_prompt", 1, 40), mask="random", seed=seed)
        self.w = w = wl.share_prompts(wl.generate(cfg, spare_pages=120), [5, 1, 6])
        self.bt = bt = DecodeBatch.from_workload(w)
        self.masked, self.hq, self.hkv, self.d = masked, 8, 2, 128
        used = w["page_table"][w["page_table"] >= 0]
        self.pool = PagePool(w["num_pages"], used)
        # a program that goes on decoding: room in the tables, bounds above the present lengths
        room = np.full((bt.batch, 8), -1, dtype=np.int32)
        bt.page_table = torch.cat([bt.page_table, torch.as_tensor(room, device="cuda")], dim=1).contiguous()
        bt.dims.max_pages_per_req = bt.page_table.shape[1]
        bt.ws = dsa.alloc_workspace(bt.dims)
        self.shared = bt.share_prefix(w["group_start"], w["prefix_len"], max_suffix=200)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.norm = dsa.make_qk_norm("rms", 1e-6, (1 + 0.2 * self.randn(128)).to(BF), (1 + 0.2 * self.randn(128)).to(BF))
        self.inv = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
        self.rope = dsa.make_rope(self.inv, [0] * 64)
        self.qkv = torch.zeros(bt.batch, 12, 128, dtype=BF, device="cuda")
        self.start = torch.empty(bt.batch + 1, dtype=torch.int32, device="cuda")
        self.slot = torch.empty(bt.batch, dtype=torch.int32, device="cuda")
        self.pos = torch.empty(bt.batch, dtype=torch.int32, device="cuda")
        self.k_rot = torch.empty(bt.batch, 2, 128, dtype=BF, device="cuda")
        self.out = torch.empty_like(bt.q)
        self.L = w["seq_len"].copy()

    def run(self, stream=None):
        bt, d = self.bt, self.bt.dims
        bt.seq_len.add_(1)
        dsa.dsa_assign_pages(d, bt.seq_len, None, self.pool.free, self.pool.count, self.pool.count, bt.page_table,
                             self.start, self.slot, self.pos, bt.ws, stream)
        dsa.dsa_qk_norm_rope(d, self.norm, self.rope, self.pos[:, None], self.qkv[:, :8], self.qkv[:, 8:10], bt.q,
                             self.k_rot, stream)
        bt.write_rows(self.slot, self.k_rot, self.qkv[:, 10:], stream)
        if self.masked:
            bt.decode_sparse_masked_shared(self.shared, self.out, stream=stream)
        else:
            bt.decode_dense_shared(self.shared, self.out, stream=stream)

    def rows(self, t, b):
        j = np.arange(self.L[b])
        table = self.bt.page_table[b].cpu().numpy()
        assert (table[j // 16] >= 0).all()
        return t[torch.as_tensor(table[j // 16].astype(np.int64)), torch.as_tensor(j % 16)]

    def check(self):
        bt, w = self.bt, self.w
        self.L = self.L + 1
        assert dsa.dsa_get_device_error(bt.ws) == 0
        assert np.array_equal(self.pos.cpu().numpy(), self.L - 1)
        # the step's q and the k row as they should be
        def turned(x, weight):
            x = x.double()
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.double()
            angle = torch.as_tensor(self.L - 1, device="cuda").double()[:, None] * torch.tensor(
                self.inv, dtype=torch.float64, device="cuda")
            c, s = angle.cos()[:, None], angle.sin()[:, None]
            a, b = x[..., :64], x[..., 64:]
            return torch.cat([a * c - b * s, b * c + a * s], -1), (a.abs() + b.abs()).repeat(1, 1, 2) * 2.0 ** -18
        for got, x, weight in ((bt.q, self.qkv[:, :8], self.norm.tensors[0]), (self.k_rot, self.qkv[:, 8:10],
                                                                              self.norm.tensors[1])):
            want, tol = turned(x, weight)
            assert ((got.double() - want).abs() <= U * want.abs() + 2 * tol).all()
        for b in range(bt.batch):
            n = int(self.L[b])
            k, v = self.rows(bt.k_pages, b), self.rows(bt.v_pages, b)
            assert torch.equal(k[-1], self.k_rot[b]) and torch.equal(v[-1], self.qkv[b, 10:])
            on = np.ones((2, n), bool)
            if self.masked:
                o = n - 1 - np.arange(n)
                P, W = int(w["prompt_len"][b]), int(w["window"][b])
                for h in range(2):
                    kept = set(wl.bits_to_offsets(w["keep_mask"][b, h]))
                    on[h] = [(n - 1 - x < P) or x == 0 or (1 <= x <= W and x in kept) for x in o]
            on = torch.as_tensor(on, device="cuda")
            q = bt.q[b].double().view(2, 4, 128)
            x = torch.einsum("hgd,nhd->hgn", q, k.double()) / math.sqrt(128)
            x = x.masked_fill(~on[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            a = torch.exp(x - z[..., None])
            want = torch.einsum("hgn,nhd->hgd", a, v.double())
            S = int(w["prefix_len"][b])
            size = torch.einsum("hgn,nhd->hgd", a[..., :S], v[:S].double().abs())
            tol = U * (want.abs() + size) + 2.0 ** -12 * v.abs().max().double()
            assert ((self.out[b].double().view(2, 4, 128) - want).abs() <= tol).all(), b
            assert (bt.lse[b].double() - z.reshape(-1)).abs().max() <= 1e-4


@pytest.mark.parametrize("masked", [False, True])
def test_steps(masked):
    """Twenty steps: pages end and begin, the free list shrinks by what was taken."""
    st = Step(masked)
    free = int(st.pool.count)
    before = (st.bt.page_table >= 0).sum()
    for i in range(20):
        st.qkv.copy_(st.randn(*st.qkv.shape).to(BF))
        st.run()
        st.check()
    assert free - int(st.pool.count) == int((st.bt.page_table >= 0).sum() - before) > 0


@pytest.mark.parametrize("masked", [False, True])
def test_steps_replayed(masked):
    """The step recorded once and replayed: every replay is a step."""
    st = Step(masked)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dsa.dsa_graph_begin(s)
    with torch.cuda.stream(s):
        st.run(s)
    g = dsa.dsa_graph_end(s)
    for i in range(20):
        st.qkv.copy_(st.randn(*st.qkv.shape).to(BF))
        torch.cuda.synchronize()
        g.launch(s)
        s.synchronize()
        st.check()
    g.close()


def test_pool_takes_back_and_gives_again():
    """Steps with a short window: pages behind it return to the pool and are used again, so that many
    more rows are decoded than the pool ever held."""
    cfg = wl.scaled(wl.WORKLOADS["llamagen-xl"], batch=3, prompt=(20, 20), seq=("after_prompt", 60, 70), mask="random",
                    window_rows=None, window=24, hq=2, hkv=2)
    w = wl.generate(cfg, spare_pages=6)
    bt = DecodeBatch.from_workload(w)
    width = 64
    table = np.full((3, width), -1, dtype=np.int32)
    table[:, :w["page_table"].shape[1]] = w["page_table"]
    bt.page_table = torch.as_tensor(table, device="cuda")
    bt.dims.max_pages_per_req = width
    bt.dims.max_kept = 80
    bt.ws = dsa.alloc_workspace(bt.dims)
    pool = PagePool(w["num_pages"], table[table >= 0])
    zero = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    L = w["seq_len"].copy()
    for i in range(400):
        bt.seq_len.add_(1)
        L += 1
        pool.evict(bt)
        _, slot, pos = pool.assign(bt)
        bt.write_rows(slot, zero + i, zero - i)
        bt.check()
        assert np.array_equal(pos.cpu().numpy(), L - 1) and int(slot.min()) >= 0
        t = bt.page_table.cpu().numpy()
        ids = np.concatenate([t[t >= 0], pool.free[:int(pool.count)].cpu().numpy()])
        assert sorted(ids) == list(range(w["num_pages"]))  # every page is somewhere, once
    out, lse = bt.decode_sparse_masked_shared(bt.share_prefix([0, 1, 2, 3], [0, 0, 0], max_suffix=80))
    want, wl_ = bt.decode_sparse_masked()
    bt.check()
    assert (out.float() - want).abs().max() <= U * want.abs().max() and (lse - wl_).abs().max() < 1e-4
