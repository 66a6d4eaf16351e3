"""Decode attention for requests that share prefixes, against softmax in 64 bits over each request's
own rows.

Bars (u = half a step of a type, bf16 2^-8, relative): the output rounds once, u |o|; the softmax
weights of the shared rows round once to bf16, so the output is off by at most u * sum a |v| over
those rows, with a the weights; the fp32 arithmetic below (scores of magnitude <= 64 with 64-128
terms off by 128 * 2^-24 * 64, 2^x to 2^-22, sums of <= 10^4 terms) stays under 2^-12 max |v|, as
for the other decode calls.  lse: the same score error, 1e-4.
"""
import math

import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


class Batch:
    """Requests in groups: `sizes` requests of prefix `prefix` each, `rest` rows behind it per request.
    Whole pages of a prefix are the same pages; a page that ends inside it is copied per request."""

    def __init__(self, sizes, prefix, rest, hkv, g, d, masked=None, seed=0, spare=4, scale=None, first_page=0):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.start = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
        B = self.B = int(self.start[-1])
        of = np.repeat(np.arange(len(sizes)), sizes)
        self.S = np.asarray(prefix, dtype=int)[of]
        self.L = self.S + np.asarray(rest, dtype=int)
        self.hkv, self.g, self.d = hkv, g, d
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        pages, at, copies = [], first_page, []
        for i, n in enumerate(sizes):
            s = int(prefix[i])
            whole, part = divmod(s, 16)
            shared = list(range(at, at + whole))
            at += whole
            for b in range(self.start[i], self.start[i] + n):
                k = -(-int(self.L[b]) // 16) - whole
                pages.append(shared + list(range(at, at + k)))
                if part and b > self.start[i]:
                    copies.append((pages[self.start[i]][whole], at, part))
                at += k
        self.pool = at + spare
        ids = first_page + self.rng.permutation(self.pool - first_page)
        width = max([len(p) for p in pages] + [1]) + 1
        self.table = np.full((B, width), -1)
        for b, p in enumerate(pages):
            self.table[b, :len(p)] = ids[np.asarray(p, dtype=int) - first_page]
        self.k, self.v = (self.randn(self.pool, 16, hkv, d) for _ in range(2))
        for src, dst, part in copies:
            for t in (self.k, self.v):
                t[ids[dst - first_page], :part] = t[ids[src - first_page], :part]
        self.q = self.randn(B, hkv * g, d)
        self.masked = masked
        self.keep = None
        if masked is not None:
            W, frac, extra = masked
            self.P = self.S + self.rng.integers(0, extra + 1, size=B)
            self.W = self.rng.integers(W // 2, W + 1, size=B)
            self.words = max(1, -(-W // 32))
            bits = self.rng.random((B, hkv, self.words * 32)) < frac
            self.bits = bits
            self.maxw = W
            w = (bits.reshape(B, hkv, self.words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
            self.mask = torch.as_tensor(w.astype(np.uint32).view(np.int32), device="cuda")
        self.dev()

    def randn(self, *s):
        return torch.randn(s, generator=self.gen, device="cuda").to(BF)

    def rows(self, b, hk):
        """Whether request b keeps each of its rows for kv head hk."""
        L = int(self.L[b])
        if self.masked is None:
            return np.ones(L, bool)
        o = L - 1 - np.arange(L)
        on = self.bits[b, hk][np.minimum(np.maximum(o - 1, 0), self.words * 32 - 1)]
        return (np.arange(L) < self.P[b]) | (o == 0) | ((o >= 1) & (o <= self.W[b]) & on)

    def most_rest(self):
        return max(int(self.rows(b, h).sum()) - int(self.S[b]) for b in range(self.B)
                   for h in (range(self.hkv) if self.masked else [0]))

    def dev(self, bound=1):
        W = self.maxw if self.masked else 0
        self.dims = dsa.make_dims(self.B, self.hkv * self.g, self.hkv, self.d, self.pool, self.table.shape[1], W,
                                  self.words if self.masked else 1, 1, "bf16", "bf16")
        self.pt, self.lens, self.pre = i32(self.table), i32(self.L), i32(self.S)
        self.gs = i32(self.start)
        self.shared = dsa.shared_prefix(self.gs, self.pre, int(self.S.max(initial=0)), max(0, self.most_rest()) * bound)
        self.ws = dsa.alloc_workspace(self.dims)
        if self.masked:
            self.plen, self.win = i32(self.P), i32(self.W)

    def run(self, shared=None, q=None, out=None, lse=True, ws=None, stream=None):
        q = self.q if q is None else q
        out = torch.full_like(q, 77.0) if out is None else out
        ls = torch.full(q.shape[:2], 77.0, dtype=torch.float32, device="cuda") if lse is True else lse
        sh, ws = shared or self.shared, self.ws if ws is None else ws
        if self.masked is None:
            dsa.dsa_decode_dense_shared(self.dims, sh, q, self.k, self.v, self.pt, self.lens, self.scale, out, ls, ws,
                                        stream)
        else:
            dsa.dsa_decode_sparse_masked_shared(self.dims, sh, q, self.k, self.v, self.pt, self.lens, self.plen, self.win,
                                                self.mask, self.scale, out, ls, ws, stream)
        return out, ls

    def ref(self, b):
        """out [hq, d], lse [hq], tolerance of out, in 64 bits."""
        L = int(self.L[b])
        pages = torch.as_tensor(self.table[b, :-(-L // 16)], device="cuda")
        k, v = (t[pages].flatten(0, 1)[:L].double() for t in (self.k, self.v))
        on = torch.as_tensor(np.stack([self.rows(b, h) for h in range(self.hkv)]), device="cuda")
        q = self.q[b].double().view(self.hkv, self.g, self.d)
        x = torch.einsum("hgd,nhd->hgn", q, k) * self.scale
        x = x.masked_fill(~on[:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        a = torch.exp(x - z[..., None])
        out = torch.einsum("hgn,nhd->hgd", a, v)
        S = int(self.S[b])
        size = torch.einsum("hgn,nhd->hgd", a[..., :S], v[:S].abs())
        most = v.abs().amax(dim=(0, 2))[:, None, None]
        tol = U * (out.abs() + size) + 2.0 ** -12 * most
        return out.reshape(-1, self.d), z.reshape(-1), tol.reshape(-1, self.d)

    def check(self, out, lse, requests=None):
        worst = 0.0
        for b in range(self.B) if requests is None else requests:
            want, z, tol = self.ref(b)
            assert torch.isfinite(out[b].float()).all(), b
            diff = (out[b].double() - want).abs()
            worst = max(worst, float((diff / tol).max()))
            assert (diff <= tol).all(), (b, worst)
            if lse is not None:
                assert (lse[b].double() - z).abs().max() <= 1e-4, b
        return worst


SHAPES = [(1, 1, 64), (2, 1, 128), (5, 2, 64), (3, 2, 128), (2, 4, 64), (8, 4, 128), (1, 8, 64), (2, 8, 128)]


@pytest.mark.parametrize("masked", [None, (40, 0.4, 9)], ids=["dense", "masked"])
@pytest.mark.parametrize("hkv,g,d", SHAPES)
def test_groups(hkv, g, d, masked):
    """Groups of every kind: one request, none, many; prefixes of nothing, inside a page, of whole
    blocks; requests with and without rows of their own."""
    sizes = [1, 0, 5, 1, 7, 2, 33]
    prefix = [0, 9, 37, 16, 128, 129, 300]
    rng = np.random.default_rng(hkv * g + d)
    rest = rng.integers(0, 90, size=sum(sizes))
    rest[0] = 1
    rest[2] = 0
    rest[8:10] = [0, 1]
    bt = Batch(sizes, prefix, rest, hkv, g, d, masked, seed=g + d)
    out, lse = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 0
    bt.check(out, lse)
    again, lse2 = bt.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    none, _ = bt.run(lse=None)
    assert torch.equal(out, none)


@pytest.mark.parametrize("S", [1, 15, 16, 17, 127, 128, 129, 255, 256, 1000, 5003])
@pytest.mark.parametrize("g,d,n", [(4, 128, 8), (1, 64, 3), (8, 64, 40)])
def test_prefix_lengths(S, g, d, n):
    bt = Batch([n], [S], [i % 3 for i in range(n)], 2, g, d, seed=S)
    bt.check(*bt.run())
    assert dsa.dsa_get_device_error(bt.ws) == 0


@pytest.mark.parametrize("rest", [1, 63, 64, 65, 700, 2500])
@pytest.mark.parametrize("masked", [None, (900, 0.9, 0), (0, 0.5, 30), (1000, 0.0, 1)])
def test_rest_lengths(rest, masked):
    """Rows behind the prefix in one chunk and in several; a bound far above the rows."""
    r = [rest, max(1, rest // 2), 1]
    bt = Batch([2, 1], [50, 7], r, 3, 4, 128, masked, seed=rest)
    out, lse = bt.run()
    bt.check(out, lse)
    bt.dev(bound=7)
    bt.check(*bt.run())
    assert dsa.dsa_get_device_error(bt.ws) == 0


def test_one_request_one_row():
    bt = Batch([1], [1], [0], 1, 1, 64)
    out, lse = bt.run()
    bt.check(out, lse)
    assert torch.equal(out[0, 0], bt.v[bt.table[0, 0], 0, 0])
    bt = Batch([1], [0], [1], 1, 1, 64)
    bt.check(*bt.run())


def test_nothing_shared():
    """max_prefix 0: no groups have to be given."""
    bt = Batch([1] * 5, [0] * 5, [40, 1, 130, 7, 16], 2, 4, 64, seed=3)
    none = dsa.shared_prefix(i32([0]), bt.pre, 0, 130)
    assert none.groups == 0
    bt.check(*bt.run(none))
    assert dsa.dsa_get_device_error(bt.ws) == 0


def test_many_groups():
    """More groups than a CTA has threads, most of a request or two."""
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 3, size=500)
    prefix = rng.integers(0, 200, size=500)
    prefix[::3] = 0
    bt = Batch(list(sizes), list(prefix), rng.integers(1, 40, size=int(sizes.sum())), 2, 2, 64, seed=5)
    bt.check(*bt.run(), requests=range(0, bt.B, 7))
    assert dsa.dsa_get_device_error(bt.ws) == 0


@pytest.mark.parametrize("hkv,g,d", [(3, 4, 128), (5, 2, 64), (1, 8, 128), (2, 1, 128)])
def test_long_and_short_prefixes(hkv, g, d):
    """Groups of several tiles and of few, prefixes of many blocks beside short ones; then with bounds
    far above them, as of prefixes that the L2 does not hold."""
    sizes, prefix = [3, 40, 1, 70, 9, 2], [5003, 1500, 2049, 1024, 700, 8]
    bt = Batch(sizes, prefix, [(7 * i) % 50 for i in range(sum(sizes))], hkv, g, d, seed=hkv + d)
    some = [0, 2, 3, 17, 42, 43, 44, 80, 113, 114, 122, 123, 124]
    out, lse = bt.run()
    bt.check(out, lse, requests=some)
    assert dsa.dsa_get_device_error(bt.ws) == 0 and torch.isfinite(out.float()).all()
    bt.table = np.pad(bt.table, ((0, 0), (0, 4000)), constant_values=-1)
    bt.dev()
    bt.shared.max_prefix = 60000
    out, lse = bt.run()
    bt.check(out, lse, requests=some)
    assert dsa.dsa_get_device_error(bt.ws) == 0 and torch.isfinite(out.float()).all()


def test_sharing_is_decode_over_own_rows():
    """The same batch with nothing shared: both within their bars, and lse equal to rounding."""
    bt = Batch([6, 3], [400, 90], [30] * 9, 4, 4, 128, seed=8)
    out, lse = bt.run()
    alone = dsa.shared_prefix(i32(np.arange(10)), i32([0] * 9), 0, 430)
    out1, lse1 = bt.run(alone)
    bt.check(out, lse)
    bt.check(out1, lse1)
    assert (lse - lse1).abs().max() < 1e-5


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_scales(scale):
    bt = Batch([5], [200], [20] * 5, 2, 4, 128, seed=2, scale=scale)
    out, lse = bt.run()
    if scale == 3.0:  # scores of some hundreds: off in proportion
        for b in range(5):
            want, z, tol = bt.ref(b)
            assert ((out[b].double() - want).abs() <= tol + 2e-3 * bt.v.abs().max()).all()
    else:
        bt.check(out, lse)


def test_sink_rows_and_rising_scores():
    """Scores that rise along the prefix (the reference moves block by block) and a first row that
    takes nearly all of the weight."""
    bt = Batch([9], [900], [33] * 9, 2, 4, 128, seed=12)
    pages = torch.as_tensor(bt.table[0, :56], device="cuda")
    q = bt.q.float().mean(dim=(0, 1))
    ramp = torch.linspace(0, 1, 896, device="cuda").view(56, 16, 1, 1) * q * 3
    bt.k[pages] = (bt.k[pages].float() + ramp).to(BF)
    bt.check(*bt.run())
    bt.k[pages[0], 0] = (q * 12).to(BF)
    bt.check(*bt.run())


def test_rows_that_nobody_keeps():
    """NaN, infinities and huge values behind the prefix in its last page, in slots without a row
    and in other requests' rows reach nobody; a row of the prefix reaches all of its group, a row of
    a request that request."""
    bt = Batch([4, 3], [37, 200], [20, 0, 5, 9, 11, 0, 40], 2, 4, 64, seed=21)
    out, lse = bt.run()
    used = np.zeros((bt.pool, 16), bool)
    for b in range(bt.B):
        j = np.arange(bt.L[b])
        used[bt.table[b, j // 16], j % 16] = True
    dead = torch.as_tensor(~used, device="cuda")
    for bad in (math.nan, math.inf, -3e38):
        for t in (bt.k, bt.v):
            t[dead] = bad
        o2, l2 = bt.run()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    # the first request's own rows share its copy of the prefix's last page
    keep = bt.v.clone()
    bt.v[bt.table[0, 37 // 16], 37 % 16:] = math.nan
    bt.v[bt.table[4, 200 // 16], 200 % 16:] = math.nan
    o2, l2 = bt.run()
    others = [1, 2, 3, 5, 6]
    assert torch.equal(out[others], o2[others]) and torch.equal(lse, l2)
    assert torch.isnan(o2[[0, 4]].float()).all()
    bt.v.copy_(keep)
    bt.v[bt.table[0, 1], 3, 1, 5] = math.nan
    o2, _ = bt.run()
    hit = torch.isnan(o2.float())
    want = torch.zeros_like(hit)
    want[:4, 4:, 5] = True
    assert torch.equal(hit, want)


def test_large_pools():
    """Pages whose bytes lie past 2^32."""
    bt = Batch([3], [150], [40, 1, 0], 32, 1, 128, seed=6, spare=1, first_page=33000)
    assert bt.k.numel() * 2 > 2**32 and bt.table[bt.table >= 0].min() >= 33000
    bt.check(*bt.run())


# ---------------------------------------------------------------------------
# invalid data: flagged, NaN where the request is invalid, the others as they were
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("masked", [None, (40, 0.4, 9)], ids=["dense", "masked"])
@pytest.mark.parametrize("what", ["len0", "len", "prefix<0", "prefix>max", "prefix>rows", "other prefix", "no prefix",
                                  "rest", "page", "rest page"])
def test_invalid_requests(what, masked):
    bt = Batch([4, 3], [64, 40], [30] * 7, 2, 4, 128, masked, seed=31)
    out, lse = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 0
    b, codes = 5, (15,)
    if what == "len0":
        bt.lens[b], codes = 0, (1,)
    elif what == "len":
        bt.lens[b], codes = 16 * bt.table.shape[1] + 1, (1,)
    elif what == "prefix<0":
        bt.pre[b] = -1
    elif what == "prefix>max":
        bt.pre[b] = 65
    elif what == "prefix>rows":
        bt.lens[b] = 39
    elif what == "other prefix":
        bt.pre[b] = 41
    elif what == "no prefix":
        bt.pre[b] = 0
        bt.shared = dsa.shared_prefix(bt.gs, bt.pre, 64, 100)
    elif what == "rest":
        bt.shared = dsa.shared_prefix(bt.gs, bt.pre, 64, bt.most_rest())
        if masked:
            bt.plen[b] = int(bt.P[b])
            bt.shared = dsa.shared_prefix(bt.gs, bt.pre, 64, max(0, int(min(bt.rows(b, h).sum() for h in range(2))) - 41))
        else:
            bt.lens[b] = int(bt.L[b]) + 1
    elif what == "page":
        bt.pt[4, 1], codes = bt.pool, (4,)  # read for the whole group
    elif what == "rest page":
        bt.pt[b, 64 // 16], codes = -1, (4,)
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) in codes
    if what == "page":
        good = [0, 1, 2, 3]
    elif what == "rest" and masked:
        good = []
    else:
        good = [0, 1, 2, 3, 4, 6]
    assert torch.equal(out[good], o2[good]) and torch.equal(lse[good], l2[good])
    if what not in ("page", "rest page", "no prefix", "rest") or (what == "rest" and not masked):
        assert torch.isnan(o2[b].float()).all() and torch.isnan(l2[b]).all()


@pytest.mark.parametrize("starts", [[1, 4, 7], [0, 4, 6], [0, 8, 7], [0, -1, 7], [0, 4, 9], [3, 2, 1]])
def test_invalid_groups(starts):
    """group_start that is no partition: flagged, and nothing outside the buffers is touched; requests
    of sound groups that no wrong one claims keep their results."""
    bt = Batch([4, 3], [64, 40], [30] * 7, 2, 4, 128, seed=31)
    bt.run()
    gs = bt.gs.clone()
    bt.gs.copy_(i32(starts))
    bt.run()
    assert dsa.dsa_get_device_error(bt.ws) in (14, 15)
    bt.gs.copy_(gs)
    bt.ws.zero_()
    bt.check(*bt.run())


def test_after_an_invalid_call():
    """A call that set an error leaves nothing behind: a prefix whose states it computed for a request
    that did not take it up is not found by the next call, which computes none."""
    bt = Batch([4, 3], [64, 40], [30] * 7, 2, 4, 128, seed=33)
    pre, gs = bt.pre.clone(), bt.gs.clone()
    out, lse = bt.run()
    bt.pre[5] = 0
    bt.run(dsa.shared_prefix(bt.gs, bt.pre, 64, 100))
    assert dsa.dsa_get_device_error(bt.ws) == 15
    dsa.dsa_clear_device_error(bt.ws)
    bt.pre.copy_(pre)
    bt.gs.copy_(i32([0, 8, 7]))
    o2, _ = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 14 and torch.isnan(o2.float()).all()
    dsa.dsa_clear_device_error(bt.ws)
    bt.gs.copy_(gs)
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 0 and torch.equal(o2, out) and torch.equal(l2, lse)


def test_groups_that_overlap():
    """Many groups that each claim the whole batch, more than any partition could have: no prefix is
    computed, every request that states one gets NaN."""
    bt = Batch([1, 60], [0, 640], [30] * 61, 2, 8, 64, seed=9)
    out, lse = bt.run()
    claim = dsa.shared_prefix(i32([0, 61] * 700 + [61]), bt.pre, 640, 40)
    o2, l2 = bt.run(claim)
    assert dsa.dsa_get_device_error(bt.ws) == 14
    assert torch.isnan(o2[1:].float()).all() and torch.isnan(l2[1:]).all() and torch.equal(o2[0], out[0])
    bt.ws.zero_()
    o2, l2 = bt.run()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_bounds_far_above():
    """max_suffix of any size plans for what the tables hold."""
    bt = Batch([3], [50], [9, 70, 0], 2, 4, 128, seed=10)
    bt.shared.max_suffix = 2**31 - 1
    bt.check(*bt.run())


# ---------------------------------------------------------------------------
# streams, graphs, steps
# ---------------------------------------------------------------------------

def test_back_to_back_calls_see_their_inputs():
    """Each call reads the q, lengths and rows that the kernels before it wrote, with nothing
    waited for in between."""
    bt = Batch([20, 12], [500, 90], np.arange(32) * 9 % 150 + 20, 4, 4, 128, seed=40)
    qs = [bt.randn(*bt.q.shape) for _ in range(6)]
    ks = [bt.randn(*bt.k.shape) for _ in range(2)]
    q, want = torch.empty_like(bt.q), []
    k = bt.k
    for i in range(12):
        torch.cuda.synchronize()
        bt.k = ks[i % 2].clone()
        want.append([x.clone() for x in bt.run(q=qs[i % 6].clone())])
    bt.k = k
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        q.copy_(qs[i % 6])
        k.copy_(ks[i % 2])
        got.append([x.clone() for x in bt.run(q=q)])
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_streams_side_by_side():
    bt = Batch([20, 12], [700, 90], [100] * 32, 2, 4, 128, seed=41)
    out, lse = bt.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    wss = [dsa.alloc_workspace(bt.dims) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            got.append(bt.run(ws=wss[i % 3]))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("masked", [None, (40, 0.4, 9)], ids=["dense", "masked"])
def test_captured_and_replayed(masked):
    bt = Batch([9, 4], [300, 33], [70] * 13, 2, 4, 128, masked, seed=42)
    out, lse = bt.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    dsa.dsa_graph_begin(s)
    bt.run(out=o2, lse=l2, stream=s)
    bt.run(out=o2, lse=l2, stream=s)
    g = dsa.dsa_graph_end(s)
    for _ in range(3):
        o2.zero_()
        torch.cuda.synchronize()
        g.launch(s)
        s.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    # new lengths and q in the same buffers
    bt.L = bt.L - 3
    bt.lens.copy_(i32(bt.L))
    bt.q.copy_(bt.randn(*bt.q.shape))
    torch.cuda.synchronize()
    g.launch(s)
    s.synchronize()
    bt.check(o2, l2)
    g.close()
