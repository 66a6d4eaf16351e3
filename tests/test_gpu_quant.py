"""The 8-bit K/V cache on the GPU: writing (bit-exact against a 64-bit restatement),
reading back (exact), and attention over it against the fp64 oracle on the
dequantised rows.

Bars of attention, from the roundings between exact inputs and the output (u = half a
step of a type: bf16 2^-8, fp16 2^-11, relative):
  bf16 q: the output rounds once (2^-8 |o|), the softmax weights once to fp16 (2^-11 of
  sum a |v| <= max |v|); the fp32 arithmetic below them (scores of magnitude <= 32 with
  64-128 terms, 2^x to 2^-22, sums of <= 10^4 terms) stays under 2^-13 max |v|.
  fp32 q: q and the weights keep 22 bits, so only that last kind is left: a score is
  off by at most 128 * 2^-24 * |q||k| / sqrt(d), below 2e-5 for the rows here, and the
  output by that times max |v| twice over (numerator and sum).
  lse: the same score error, 1e-4 as for the other decode calls; a score of thousands is
  moreover off in proportion to itself: 2^-22 by the halves of an fp32 q (11 bits each,
  half a step of the second), and 2^-24 for each of scale, log2 e, their product, the
  row's factor, the sum, its product, the reference and the change of base: 2^-21
  for these eight, so less than 2^-20 |lse| together.
"""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_serving_gb300 import dsa
from kv_cache_serving_gb300 import workloads as wl
from kv_cache_serving_gb300.session import DecodeBatch, QuantBatch

pytestmark = pytest.mark.gpu

LSE_MAX = 1e-4
SENTINEL = -12345.0
E_MIN, E_MAX = -40, 40


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


# ---------------------------------------------------------------------------
# 64-bit restatement of the format
# ---------------------------------------------------------------------------

def e4m3_table():
    """Value of every code byte."""
    u = np.arange(256)
    ex, man = (u >> 3) & 15, u & 7
    val = np.where(ex > 0, (8 + man) * 2.0 ** (ex - 10.0), man * 2.0 ** -9)
    val = np.where((u & 127) == 127, np.nan, val)
    return np.where(u >= 128, -val, val)


TABLE = e4m3_table()
POSITIVE = TABLE[:127]  # 0 .. 448, ascending


def nearest_code(x):
    """Code byte of the e4m3 value nearest to x (fp64), ties to the even code,
    saturated; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.searchsorted(POSITIVE, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = pick + np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def exponent_for(a):
    e = E_MIN
    while e < E_MAX and a > 448.0 * 2.0 ** e:
        e += 1
    return e


class RefCache:
    """The cache as numpy arrays, written row block by row block."""

    def __init__(self, pages, hkv, d):
        self.codes = {x: np.zeros((pages, hkv, 16, d), np.uint8) for x in "kv"}
        self.scale = {x: np.ones((pages, hkv)) for x in "kv"}

    def write(self, new, table, L, n):
        for b in range(len(L)):
            first = int(L[b]) - int(n[b])
            for p in range(first // 16, (int(L[b]) - 1) // 16 + 1) if n[b] else ():
                lo, hi = max(first, 16 * p), min(int(L[b]), 16 * p + 16)
                page, at = table[b, p], lo - 16 * p
                for x in "kv":
                    rows = new[x][b, lo - first:hi - first].double().numpy()
                    for h in range(rows.shape[1]):
                        r = rows[:, h]
                        a = np.abs(r[np.isfinite(r)]).max(initial=0.0)
                        e = exponent_for(a)
                        if at > 0:
                            was = int(np.log2(self.scale[x][page, h]))
                            e = max(e, was)
                            old = TABLE[self.codes[x][page, h, :at]] * 2.0 ** (was - e)
                            if e > was:
                                keep = np.signbit(old) & (old == 0)
                                self.codes[x][page, h, :at] = np.where(
                                    keep, 128, nearest_code(old))
                        self.codes[x][page, h, at:at + len(r)] = nearest_code(r * 2.0 ** -e)
                        self.scale[x][page, h] = 2.0 ** e


def nan_equal_codes(a, b):
    """Equal bytes, any NaN code for a NaN code."""
    return np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b)


class Pool:
    """A paged 8-bit cache of its own on the GPU, for the write and read calls."""

    def __init__(self, batch, hkv, d, dtype, max_pages, spare=2, seed=0):
        rng = np.random.default_rng(seed)
        self.pages = batch * max_pages + spare
        self.table = rng.permutation(self.pages)[:batch * max_pages].reshape(batch, max_pages)
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.dims = dsa.make_dims(batch, hkv, hkv, d, self.pages, max_pages, 0, 1, 1, dtype, dtype)
        self.ws = dsa.alloc_workspace(self.dims)
        fill = torch.as_tensor(rng.integers(0, 120, (self.pages, hkv, 16, d)).astype(np.uint8))
        self.k, self.v = fill.clone().cuda(), fill.flip(0).clone().cuda()
        self.ks, self.vs = (torch.ones(self.pages, hkv, device="cuda") for _ in range(2))
        self.cache = dsa.quant_cache(self.k, self.v, self.ks, self.vs)
        self.ref = RefCache(self.pages, hkv, d)
        self.ref.codes = {"k": fill.numpy().copy(), "v": fill.flip(0).numpy().copy()}
        self.pt = torch.as_tensor(self.table.astype(np.int32)).cuda()

    def write(self, kn, vn, L, n, device_n=True):
        dev = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
        dsa.dsa_quant_write(self.dims, self.cache, kn.cuda(), vn.cuda(), self.pt, dev(L),
                            dev(n) if device_n else None, self.ws)
        torch.cuda.synchronize()
        return dsa.dsa_get_device_error(self.ws)

    def check(self):
        for t, s, x in ((self.k, self.ks, "k"), (self.v, self.vs, "v")):
            got, want = nan_equal_codes(t.cpu().numpy(), self.ref.codes[x])
            assert np.array_equal(s.cpu().numpy().astype(np.float64), self.ref.scale[x])
            assert np.array_equal(got, want)


def rows(rng, shape, dt, spread=3.0):
    x = rng.standard_normal(shape) * 2.0 ** rng.uniform(-spread, spread, shape[:2] + (1, 1))
    return torch.as_tensor(x).to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_write_bit_exact(d, hkv, dtype):
    """A ragged prompt, then single rows across page borders, then ragged chunks that
    start inside pages: every code and scale of the pool, untouched slots included."""
    rng = np.random.default_rng(d + hkv)
    B, mp = 4, 7
    pool = Pool(B, hkv, d, dtype, mp, seed=hkv)
    L = np.array([1, 15, 16, 37])
    new = {x: rows(rng, (B, 37, hkv, d), pool.dt) for x in "kv"}
    assert pool.write(new["k"], new["v"], L, L) == 0
    pool.ref.write(new, pool.table, L, L)
    pool.check()
    for step in range(18):  # one row each; sizes grow, so scales have to move
        L = L + 1
        new = {x: rows(rng, (B, 1, hkv, d), pool.dt, 2.0 + step / 3) for x in "kv"}
        assert pool.write(new["k"], new["v"], L, np.ones(B, int), device_n=step % 2 == 0) == 0
        pool.ref.write(new, pool.table, L, np.ones(B, int))
    pool.check()
    n = np.array([0, 5, 17, 33])
    L = L + n
    new = {x: rows(rng, (B, 33, hkv, d), pool.dt, 6.0) for x in "kv"}
    assert pool.write(new["k"], new["v"], L, n) == 0
    pool.ref.write(new, pool.table, L, n)
    pool.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_special_values(dtype):
    """Zeros of both signs, infinities, NaN, the largest and smallest magnitudes, and
    values on the border between two codes."""
    pool = Pool(1, 4, 64, dtype, 3)
    x = torch.zeros(1, 40, 4, 64, dtype=torch.float64)
    x[0, :, 0] = -0.0                                            # head 0: zeros alone
    x[0, :16, 1] = torch.linspace(-500, 500, 64).double()          # over 448: the scale is 2
    x[0, 0, 1, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    x[0, 16:, 1] = 3e38
    x[0, :, 2] = 1e-38                                           # below every scale
    ties = torch.as_tensor((POSITIVE[:-1] + POSITIVE[1:]) / 2)[-64:]
    x[0, :, 3] = ties                                            # halfway between codes
    x[0, 3, 3] = -ties
    x = x.to(pool.dt)
    assert pool.write(x, -x, [40], [40]) == 0
    pool.ref.write({"k": x, "v": -x}, pool.table, [40], [40])
    pool.check()


def test_write_strided_rows():
    """K and V as slices of one fused projection."""
    rng = np.random.default_rng(5)
    pool = Pool(2, 2, 128, "bf16", 3)
    qkv = rows(rng, (2, 20, 10, 128), torch.bfloat16).cuda()
    k, v = qkv[:, :, 6:8], qkv[:, :, 8:10]
    L = np.array([20, 33])
    assert pool.write(k, v, L, [20, 20]) == 0
    # the page before request 1's rows was never written: its scale of one stays
    pool.ref.write({"k": k.cpu(), "v": v.cpu()}, pool.table, L, [20, 20])
    pool.check()


def test_write_flags_bad_requests():
    """A bad length, count, page id or old scale: flagged, nothing written for it, the
    other requests written."""
    rng = np.random.default_rng(6)
    cases = [((0, 5), (1, 1), None, 1), ((99, 5), (1, 1), None, 1), ((5, 5), (-1, 1), None, 11),
             ((5, 5), (6, 1), None, 11), ((3, 5), (4, 1), None, 11),
             ((17, 5), (1, 1), "page", 4), ((5, 5), (1, 1), "scale", 12)]
    for L, n, what, code in cases:
        pool = Pool(2, 1, 64, "f32", 2)
        if what == "page":
            pool.pt[0, 1] = pool.pages
        if what == "scale":
            pool.ks[pool.table[0, 0]] = 3.0
            pool.vs[pool.table[0, 0]] = 0.0
        before = [t.clone() for t in (pool.k, pool.v, pool.ks, pool.vs)]
        new = {x: rows(rng, (2, 5, 1, 64), torch.float32) for x in "kv"}
        assert pool.write(new["k"], new["v"], L, n) == code
        other = torch.as_tensor([p for p in range(pool.pages) if p not in pool.table[1]]).cuda()
        for t, b in zip((pool.k, pool.v, pool.ks, pool.vs), before):
            assert torch.equal(t[other], b[other])
        assert not torch.equal(pool.k[pool.table[1, 0]], before[0][pool.table[1, 0]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_read_exact(d, dtype):
    rng = np.random.default_rng(d)
    B, hkv, mp = 4, 3, 6
    pool = Pool(B, hkv, d, dtype, mp)
    exps = rng.integers(E_MIN, E_MAX + 1, (pool.pages, hkv))
    pool.ks.copy_(torch.as_tensor(2.0 ** exps).float())
    pool.vs.copy_(torch.as_tensor(2.0 ** -exps).float())
    codes = rng.integers(0, 256, (pool.pages, hkv, 16, d)).astype(np.uint8)
    pool.k.copy_(torch.as_tensor(codes))
    L = np.array([96, 33, 1, 50])
    start, n = np.array([7, 16, 0, 49]), np.array([60, 17, 1, 0])
    dev = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    ko = torch.full((B, 60, hkv, d), SENTINEL, dtype=pool.dt, device="cuda")
    vo = torch.full_like(ko, SENTINEL)
    dsa.dsa_quant_read(pool.dims, pool.cache, pool.pt, dev(L), dev(start), dev(n), ko, vo, pool.ws)
    assert dsa.dsa_get_device_error(pool.ws) == 0
    ko2 = torch.full_like(ko, SENTINEL)
    dsa.dsa_quant_read(pool.dims, pool.cache, pool.pt, dev(L), dev(start), dev(n), ko2, None,
                       pool.ws)
    assert torch.equal(ko.view(torch.uint8), ko2.view(torch.uint8))
    for out, t, s in ((ko, pool.k, pool.ks), (vo, pool.v, pool.vs)):
        want = np.full(tuple(out.shape), float(torch.tensor(SENTINEL).to(pool.dt)))
        t, s = t.cpu().numpy(), s.cpu().numpy().astype(np.float64)
        for b in range(B):
            for i in range(n[b]):
                j = start[b] + i
                pg = pool.table[b, j // 16]
                want[b, i] = TABLE[t[pg, :, j % 16]] * s[pg][:, None]
        assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)


def test_read_flags_bad_rows():
    pool = Pool(2, 1, 64, "f32", 2)
    dev = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    for L, start, n, page, code in (((0, 4), (0, 0), (1, 1), None, 1), ((4, 4), (-1, 0), (1, 1), None, 11),
                                    ((4, 4), (2, 0), (3, 1), None, 11), ((20, 4), (0, 0), (9, 1), None, 11),
                                    ((20, 4), (2**31 - 1, 0), (2, 1), None, 11),
                                    ((20, 4), (17, 0), (1, 1), -1, 4)):
        pt = pool.pt.clone()
        if page is not None:
            pt[0, 1] = page
        out = torch.full((2, 8, 1, 64), SENTINEL, device="cuda")
        dsa.dsa_quant_read(pool.dims, pool.cache, pt, dev(L), dev(start), dev(n), out, None, pool.ws)
        assert dsa.dsa_get_device_error(pool.ws) == code
        dsa.dsa_clear_device_error(pool.ws)
        assert (out[0] == SENTINEL).all() and (out[1, 1:] == SENTINEL).all()
        assert (out[1, 0] != SENTINEL).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def dequantised(qb):
    """K/V pages of the oracle's layout [pages, 16, hkv, d] as fp32 (exact)."""
    res = []
    for t, s in ((qb.k, qb.k_scale), (qb.v, qb.v_scale)):
        x = TABLE[t.view(torch.uint8).cpu().numpy()] * s.double().cpu().numpy()[:, :, None, None]
        res.append(torch.as_tensor(x.transpose(0, 2, 1, 3).astype(np.float32)).contiguous())
    return res


def compare(out, lse, ref, ref_lse, vmax, fp32):
    out = np.asarray(out, np.float64).reshape(ref.shape)
    assert np.isfinite(out).all()
    err = np.abs(out - ref)
    if fp32:
        assert (err <= 4e-5 * vmax).all(), (err.max(), vmax)
    else:
        bound = np.abs(ref) * 2.0 ** -8 + vmax * (2.0 ** -11 + 2.0 ** -13)
        assert (err <= bound).all(), (err - bound).max()
    lse = np.asarray(lse, np.float64).reshape(ref_lse.shape)
    assert (np.abs(lse - ref_lse) <= LSE_MAX + 2.0 ** -20 * np.abs(ref_lse)).all()


def case(d, g, dtype="bf16", batch=6, hkv=2, lo=1, hi=420, prompt=(0, 90), W=70, seed=0):
    return wl.Config(f"q8-{d}-{g}", batch, hkv * g, hkv, d, dtype, prompt, (8,), None, W,
                     ("abs", lo, hi), "random", band=2, seed=seed)


def run_modes(qb, w, modes=("dense", "list", "masked"), mask=None):
    """Every decode call against the oracle on the dequantised rows."""
    bt = qb.batch
    inp = dict(w)
    inp["k_pages"], inp["v_pages"] = dequantised(qb)
    if mask is not None:
        inp["keep_mask"] = mask
    table = np.asarray(w["page_table"])
    used = table[table >= 0]
    vmax = float(inp["v_pages"][torch.as_tensor(used)].abs().nan_to_num(0).max())
    got = {}
    for mode in modes:
        if mode == "list":
            bt.build_index()
        out, lse = torch.full_like(qb.out, SENTINEL), torch.full_like(qb.lse, SENTINEL)
        {"dense": qb.decode_dense, "list": qb.decode_sparse,
         "masked": qb.decode_sparse_masked}[mode](out=out, lse=lse)
        torch.cuda.synchronize()
        assert bt.device_error() == 0, mode
        ref, ref_lse = oracle.decode(inp, sparse=mode != "dense")
        compare(out.float().cpu(), lse.cpu(), ref, ref_lse, vmax, w["dtype"] == "f32")
        got[mode] = out, lse
    if "list" in got and "masked" in got:  # the same rows in the same order: the same bits
        assert torch.equal(got["list"][0], got["masked"][0])
        assert torch.equal(got["list"][1], got["masked"][1])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_every_build(d, g, dtype):
    w = wl.generate(case(d, g, dtype, seed=d + g), spare_pages=3)
    run_modes(QuantBatch.from_batch(DecodeBatch.from_workload(w)), w)


@pytest.mark.parametrize("name,batch", [("llamagen-xl", 32), ("janus-pro-7b", 9), ("emu3-8b", 3)])
def test_decode_workload_shapes(name, batch):
    w = wl.generate(wl.scaled(wl.WORKLOADS[name], batch=batch))
    run_modes(QuantBatch.from_batch(DecodeBatch.from_workload(w)), w)


@pytest.mark.parametrize("L", [1, 15, 16, 17, 63, 64, 65, 257, 5000])
def test_decode_single_request(L):
    """One request of every length class: the dense call cuts its units over CTAs, the
    sparse ones too when the kept set is long."""
    w = wl.generate(case(128, 4, batch=1, lo=L, hi=L, prompt=(0, min(L, 900)), W=90, seed=L))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    first = run_modes(qb, w)
    again = run_modes(qb, w)  # the arrival counters are back at zero: the same bits
    for mode in first:
        assert torch.equal(first[mode][0], again[mode][0])
        assert torch.equal(first[mode][1], again[mode][1])


def test_decode_many_short_requests():
    """More requests than the prefix sum has threads, lengths 1..40, past the request
    schedule's limit."""
    w = wl.generate(case(64, 2, batch=1100, hkv=2, hi=40, prompt=(0, 20), W=16, seed=3))
    run_modes(QuantBatch.from_batch(DecodeBatch.from_workload(w)), w)


@pytest.mark.parametrize("batch,hkv,g,d,lo,hi", [(3, 2, 2, 64, 1, 3), (48, 8, 1, 128, 1, 40),
                                                 (130, 8, 2, 128, 1, 165), (90, 16, 1, 64, 100, 200)])
def test_decode_dense_short_units(batch, hkv, g, d, lo, hi):
    """Dense shares of a unit or less: fewer tiles than the CTAs' least share, more units than
    resident CTAs."""
    w = wl.generate(case(d, g, batch=batch, hkv=hkv, lo=lo, hi=hi, prompt=(1, 2), W=16, seed=batch))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_modes(qb, w, ("dense",))


def test_decode_long_prompts_share_units():
    """Sparse rows of few units with long prompts: several CTAs per unit."""
    w = wl.generate(case(128, 8, batch=2, hkv=1, lo=3000, hi=4000, prompt=(1500, 2900), W=200, seed=9))
    run_modes(QuantBatch.from_batch(DecodeBatch.from_workload(w)), w)


def test_decode_window_edges():
    w = wl.generate(case(128, 2, batch=6, lo=100, hi=300, prompt=(0, 40), W=64, seed=21))
    w["window"][1] = 0
    w["keep_mask"][2] = 0
    w["keep_mask"][3] = 0xFFFFFFFF
    w["prompt_len"][4] = 1000  # longer than the request: every row is a prompt row
    w["max_kept"] = 320
    run_modes(QuantBatch.from_batch(DecodeBatch.from_workload(w)), w)


def test_decode_long_window_by_list():
    """A window past the masked call's 1024 offsets: refused there, served by lists."""
    w = wl.generate(case(64, 4, batch=3, lo=1500, hi=2200, prompt=(0, 60), W=1500, seed=11))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_modes(qb, w, modes=("dense", "list"))
    with pytest.raises(dsa.DSAError):
        qb.decode_sparse_masked()


def test_decode_scales_far_apart():
    """Pages whose V scales differ by up to 2^60: the large ones decide the output, the
    sum counts every row."""
    w = wl.generate(case(128, 4, batch=4, lo=200, hi=500, prompt=(150, 180), W=64, seed=31))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    rng = np.random.default_rng(1)
    shift = torch.as_tensor(2.0 ** rng.integers(-30, 31, tuple(qb.v_scale.shape))).float().cuda()
    qb.v_scale.copy_(shift)
    run_modes(qb, w)


@pytest.mark.parametrize("peak", [30.0, 300.0])
def test_decode_peaked_scores(peak):
    """Scores far apart (a running maximum that climbs by thousands of steps of the
    slack, and weights that vanish); q of very different sizes."""
    w = wl.generate(case(128, 4, "f32", batch=4, lo=200, hi=600, prompt=(150, 180), W=64, seed=41))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    unit = torch.ones(128, device="cuda") / 128 ** 0.5
    sizes = torch.tensor([1e-30, 1.0, peak, -peak], device="cuda")
    bt.q.copy_((unit * sizes[:, None, None]).expand_as(bt.q))
    # every element of a row the same small integer: all products and sums are exact
    n = torch.randint(0, 64, qb.k.shape[:3], device="cuda").float()
    qb.k.copy_(n[..., None].expand(qb.k.shape).to(torch.float8_e4m3fn))
    qb.k_scale.fill_(2.0 ** -4)
    w["q"] = bt.q.cpu()
    run_modes(qb, w)


def test_decode_ignores_unread_rows():
    """NaN codes in every row a call must not read, NaN scales in every page: nothing
    changes, bit for bit."""
    w = wl.generate(case(128, 4, batch=5, lo=60, hi=500, seed=51), spare_pages=4)
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    before = run_modes(qb, w)
    table, keep = np.asarray(w["page_table"]), {}
    for mode in ("dense", "masked"):
        read = np.zeros(tuple(qb.k.shape[:3]), bool)
        for b in range(w["batch"]):
            for hk in range(w["hkv"]):
                L = int(w["seq_len"][b])
                rows_ = np.arange(L) if mode == "dense" else oracle.kept_set(
                    L, int(w["prompt_len"][b]), int(w["window"][b]), w["keep_mask"][b, hk])
                read[table[b, rows_ // 16], hk, rows_ % 16] = True
        keep[mode] = torch.as_tensor(read).cuda()
    codes = [t.view(torch.uint8).clone() for t in (qb.k, qb.v)]
    scales = [t.clone() for t in (qb.k_scale, qb.v_scale)]
    for mode, names in (("dense", ("dense",)), ("masked", ("list", "masked"))):
        for t, c, s, sc in zip((qb.k, qb.v), codes, (qb.k_scale, qb.v_scale), scales):
            t.view(torch.uint8).copy_(torch.where(keep[mode][..., None], c, torch.full_like(c, 127)))
            s.copy_(torch.where(keep[mode].any(-1), sc, torch.full_like(sc, float("nan"))))
        for name in names:
            out, lse = {"dense": qb.decode_dense, "list": qb.decode_sparse,
                        "masked": qb.decode_sparse_masked}[name](out=torch.empty_like(qb.out),
                                                                 lse=torch.empty_like(qb.lse))
            torch.cuda.synchronize()
            assert qb.batch.device_error() == 0
            assert torch.equal(out, before[name][0]) and torch.equal(lse, before[name][1])


def test_decode_nan_rows_stay_nan():
    """A kept row that holds NaN makes its heads NaN, and no others."""
    w = wl.generate(case(64, 2, batch=2, hkv=2, lo=100, hi=200, prompt=(50, 60), seed=61))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    page = int(w["page_table"][0, 1])
    qb.k.view(torch.uint8)[page, 1, 3, 5] = 127
    for call in (qb.decode_dense, qb.decode_sparse_masked):
        out, _ = call()
        torch.cuda.synchronize()
        out = out.float().cpu()
        assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all()
        assert torch.isfinite(out[1]).all()


def test_decode_request_order_and_no_lse():
    w = wl.generate(case(128, 1, batch=7, hkv=4, seed=71))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    want, _ = qb.decode_sparse_masked()
    want = want.clone()
    order = torch.as_tensor(bt.longest_first_order()).cuda()
    out = torch.empty_like(want)
    for req in (None, order):
        out.fill_(0)
        dsa.dsa_decode_sparse_masked_quant(bt.dims, bt.q, qb.cache, bt.page_table, bt.seq_len,
                                           bt.prompt_len, bt.window, bt.keep_mask, bt.scale, out,
                                           None, bt.ws, request_order=req)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    dsa.dsa_decode_dense_quant(bt.dims, bt.q, qb.cache, bt.page_table, bt.seq_len, bt.scale, out,
                               None, bt.ws)
    torch.cuda.synchronize()
    assert bt.device_error() == 0


@pytest.mark.parametrize("what,code", [("seq_len", 1), ("long", 1), ("prompt", 2), ("window", 3),
                                       ("page", 4), ("scale", 12), ("order", 9)])
def test_decode_flags_bad_requests(what, code):
    """Invalid per-request data: flagged, NaN where the request itself is invalid, the
    other requests unharmed."""
    w = wl.generate(case(128, 2, batch=3, lo=100, hi=200, seed=81))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    calls = {"masked": qb.decode_sparse_masked}
    if what in ("seq_len", "long", "page", "scale"):
        calls["dense"] = qb.decode_dense
    good = {m: [t.clone() for t in c()] for m, c in calls.items()}
    order = None
    if what in ("seq_len", "long"):
        bt.seq_len[1] = 0 if what == "seq_len" else 100000
    elif what == "prompt":
        bt.prompt_len[1] = -1
    elif what == "window":
        bt.window[1] = bt.dims.max_window + 1
    elif what == "page":
        bt.page_table[1, 0] = bt.dims.num_pages
    elif what == "scale":
        qb.k_scale[bt.page_table[1, 0]] = 1.5
    elif what == "order":
        order = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    for mode, call in calls.items():
        out, lse = torch.full_like(qb.out, SENTINEL), torch.full_like(qb.lse, SENTINEL)
        call(out=out, lse=lse, **({"request_order": order} if order is not None else {}))
        assert bt.device_error() == code, mode
        dsa.dsa_clear_device_error(bt.ws)
        for b in (0, 2):
            assert torch.allclose(out[b].float(), good[mode][0][b].float(), rtol=2 ** -7, atol=2e-3)
        if code <= 3:
            assert torch.isnan(out[1].float()).all() and torch.isnan(lse[1]).all()


# ---------------------------------------------------------------------------
# several query tokens
# ---------------------------------------------------------------------------

def run_chunk(qb, w, qmax, q_len, seed=0, mask=None):
    bt = qb.batch
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(w["batch"], qmax, w["hq"], w["head_dim"], generator=gen).to(torch.bfloat16)
    out = torch.full(tuple(q.shape), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(tuple(q.shape[:3]), SENTINEL, device="cuda")
    ql = torch.as_tensor(np.asarray(q_len, np.int32)).cuda()
    qb.prefill_sparse(q.cuda(), ql, out, lse)
    torch.cuda.synchronize()
    assert bt.device_error() == 0
    inp = dict(w, q=q)
    inp["k_pages"], inp["v_pages"] = dequantised(qb)
    ref, ref_lse = oracle.multi(inp, q_len)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    stay = float(torch.tensor(SENTINEL).to(torch.bfloat16))
    for b in range(w["batch"]):
        assert (o[b, q_len[b]:] == stay).all() and (l[b, q_len[b]:] == SENTINEL).all()
    table = np.asarray(w["page_table"])
    vmax = float(inp["v_pages"][torch.as_tensor(table[table >= 0])].abs().max())
    on = ~np.isnan(ref)
    if on.any():
        compare(o[on], l[~np.isnan(ref_lse)], ref[on], ref_lse[~np.isnan(ref_lse)], vmax, False)
    return out, lse


def chunk_lens(w, qmax, seed):
    rng = np.random.default_rng(seed)
    n = np.array([int(rng.integers(0, min(qmax, int(L)) + 1)) for L in w["seq_len"]])
    n[0] = min(qmax, int(w["seq_len"][0]))
    return n


@pytest.fixture
def split(request):
    """dsa_set_prefill_split for one test: 1 whole units, n >= 2 units in n parts."""
    saved = dsa.dsa_get_prefill_split()
    dsa.dsa_set_prefill_split(request.param)
    yield request.param
    dsa.dsa_set_prefill_split(saved)


@pytest.mark.parametrize("split", [0, 1, 3], indirect=True)
@pytest.mark.parametrize("qmax", [1, 7, 16, 70])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_every_build(d, g, qmax, split):
    w = wl.generate(case(d, g, seed=d + g + qmax), spare_pages=3)
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_chunk(qb, w, qmax, chunk_lens(w, qmax, g), seed=qmax)


@pytest.mark.parametrize("name,batch,qmax", [("janus-pro-7b", 5, 32), ("llamagen-xl", 6, 24),
                                             ("emu3-8b", 2, 40)])
@pytest.mark.parametrize("split", [0, 1], indirect=True)
def test_chunk_workload_shapes(name, batch, qmax, split):
    w = wl.generate(wl.scaled(wl.WORKLOADS[name], batch=batch))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_chunk(qb, w, qmax, chunk_lens(w, qmax, 1))


@pytest.mark.parametrize("split", [0, 1], indirect=True)
def test_chunk_whole_sequences_and_edges(split):
    """Every row a query, no query, a window of 0, empty and full masks, a prompt longer
    than the request."""
    w = wl.generate(case(128, 4, batch=6, lo=30, hi=150, prompt=(0, 40), W=64, seed=5))
    L = w["seq_len"]
    w["window"][1] = 0
    w["keep_mask"][2] = 0
    w["keep_mask"][3] = 0xFFFFFFFF
    w["prompt_len"][5] = 1000
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_chunk(qb, w, int(L.max()), [int(L[0]), 0, int(L[2]), min(17, int(L[3])), 1, int(L[5])], seed=6)


@pytest.mark.parametrize("split", [0, 1], indirect=True)
def test_chunk_long_window(split):
    w = wl.generate(case(128, 2, batch=3, lo=1500, hi=2200, prompt=(0, 60), W=1500, seed=11))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    run_chunk(qb, w, 40, chunk_lens(w, 40, 12))


@pytest.mark.parametrize("qmax", [3, 16, 40])
def test_chunk_split_units(qmax):
    """One long request: the pages of its units are cut over CTAs, and a repeated call
    gives the same bits."""
    w = wl.generate(case(128, 4, batch=1, hkv=1, lo=3000, hi=3000, prompt=(2500, 2500), W=90, seed=7))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    a = run_chunk(qb, w, qmax, [qmax])
    b = run_chunk(qb, w, qmax, [qmax])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_chunk_of_one_is_a_decode_step():
    w = wl.generate(case(128, 4, batch=5, lo=50, hi=300, seed=13))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    out, lse = qb.decode_sparse_masked()
    o2, l2 = torch.empty_like(out)[:, None], torch.empty_like(lse)[:, None]
    qb.prefill_sparse(bt.q[:, None].contiguous(), torch.ones(5, dtype=torch.int32, device="cuda"),
                      o2, l2)
    torch.cuda.synchronize()
    assert torch.allclose(o2[:, 0].float(), out.float(), rtol=2 ** -7, atol=2e-3)
    assert torch.allclose(l2[:, 0], lse, atol=1e-5)


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
def test_chunk_ignores_unread_rows(split):
    w = wl.generate(case(128, 4, batch=4, lo=100, hi=400, prompt=(20, 60), W=64, seed=17), spare_pages=4)
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    n = np.minimum(9, w["seq_len"])
    want = run_chunk(qb, w, 9, n)
    table = np.asarray(w["page_table"])
    read = np.zeros(tuple(qb.k.shape[:3]), bool)
    for b in range(4):
        for hk in range(w["hkv"]):
            for t in range(int(n[b])):
                j = oracle.kept_set(int(w["seq_len"][b] - n[b] + t + 1), int(w["prompt_len"][b]),
                                    int(w["window"][b]), w["keep_mask"][b, hk])
                read[table[b, j // 16], hk, j % 16] = True
    on = torch.as_tensor(read).cuda()
    for t, s in ((qb.k, qb.k_scale), (qb.v, qb.v_scale)):
        c = t.view(torch.uint8)
        c.copy_(torch.where(on[..., None], c, torch.full_like(c, 127)))
        s.copy_(torch.where(on.any(-1), s, torch.full_like(s, float("nan"))))
    gen = torch.Generator().manual_seed(0)
    q = torch.randn(4, 9, w["hq"], 128, generator=gen).to(torch.bfloat16).cuda()
    out, lse = torch.full_like(want[0], SENTINEL), torch.full_like(want[1], SENTINEL)
    qb.prefill_sparse(q, torch.as_tensor(n.astype(np.int32)).cuda(), out, lse)
    torch.cuda.synchronize()
    assert qb.batch.device_error() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("split", [1, 2], indirect=True)
@pytest.mark.parametrize("d,n", [(64, 20), (128, 6), (128, 20)])
def test_chunk_of_16_byte_alignment(d, n, split):
    """q and out that begin 16 bytes into their memory: the same bits as whole ones."""
    w = wl.generate(case(d, 4, batch=2, hkv=2, lo=100, hi=160, prompt=(40, 60), W=64, seed=31))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    gen = torch.Generator().manual_seed(2)
    q = torch.randn(2, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    ql = torch.full((2,), n, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    qb.prefill_sparse(q, ql, out, None)
    flat = [torch.full((q.numel() + 16,), SENTINEL, dtype=q.dtype, device="cuda") for _ in range(2)]
    q2, out2 = (f[8:8 + q.numel()].view(q.shape) for f in flat)
    q2.copy_(q)
    qb.prefill_sparse(q2, ql, out2, None)
    torch.cuda.synchronize()
    assert qb.batch.device_error() == 0
    assert torch.equal(out, out2)
    edge = torch.cat([flat[1][:8], flat[1][8 + q.numel():]])
    assert (edge == torch.tensor(SENTINEL, dtype=q.dtype, device="cuda")).all()


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d,g,n", [(64, 2, 20), (128, 1, 20), (128, 4, 9), (128, 4, 40), (128, 2, 80)])
def test_chunk_queries_of_unlike_sizes(d, g, n, split):
    """A query far larger, far smaller, infinite or NaN beside others of its tile: the others
    keep their results.  Not their bits: the references of a tile may move together, and the
    weights (fp16, 2^-11 each) and the output (bf16, 2^-8 against 2^-8) are rounded anew, so
    two runs lie within 2^-7 of the value and 2 * 2^-11 of the largest |V| (about 4)."""
    w = wl.generate(case(d, g, batch=2, hkv=2, lo=200, hi=260, prompt=(40, 60), W=64, seed=29))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(2, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    ql = torch.full((2,), n, dtype=torch.int32, device="cuda")

    def run(x):
        out, lse = torch.empty_like(x), torch.empty(x.shape[:3], device="cuda")
        qb.prefill_sparse(x, ql, out, lse)
        torch.cuda.synchronize()
        assert qb.batch.device_error() == 0
        return out, lse

    out, lse = run(q)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[[2, n - 1]] = False
    for factor in (2.0 ** 24, 2.0 ** 50, 2.0 ** -50, 2.0 ** -120, float("inf"), float("nan")):
        x = q.clone()
        x[:, [2, n - 1]] *= factor
        o, l = run(x)
        assert torch.allclose(o[:, others].float(), out[:, others].float(), rtol=2 ** -7, atol=4e-3)
        assert torch.allclose(l[:, others], lse[:, others], rtol=0, atol=1e-5)
        if factor < 1:  # scores of nothing: lse is the log of the rows kept
            assert torch.allclose(l[:, ~others].exp(), l[:, ~others].exp().round(), rtol=1e-5)
        if 1 < factor < float("inf"):
            assert torch.isfinite(o).all() and torch.isfinite(l).all()


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d,g", [(64, 2), (128, 1), (128, 4)])
def test_chunk_nan_rows_reach_only_their_queries(d, g, split):
    """NaN in V (and in K) of a row of the chunk: queries before it, and queries whose mask
    skips it, keep their bits' worth; the others get the NaN where it belongs."""
    w = wl.generate(case(d, g, batch=2, hkv=2, lo=200, hi=260, prompt=(40, 60), W=64, seed=23))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt, n = qb.batch, 20
    gen = torch.Generator().manual_seed(0)
    q = torch.randn(2, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    ql = torch.full((2,), n, dtype=torch.int32, device="cuda")

    def run():
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        qb.prefill_sparse(q, ql, out, lse)
        torch.cuda.synchronize()
        assert bt.device_error() == 0
        return out.float().cpu(), lse.cpu()

    base, base_lse = run()
    for what in ("v", "k"):
        codes = (qb.v if what == "v" else qb.k).view(torch.uint8)
        for b, back in ((0, 8), (1, 30)):  # a row of the chunk, a window row before it
            j = int(w["seq_len"][b]) - 1 - back
            page = int(w["page_table"][b, j // 16])
            keepers = torch.zeros(n, dtype=torch.bool)
            for t in range(n):
                i = int(w["seq_len"][b]) - n + t
                keepers[t] = j in oracle.kept_set(i + 1, int(w["prompt_len"][b]), int(w["window"][b]),
                                                  w["keep_mask"][b, 1]) if i >= j else False
            assert keepers.any() and not keepers.all()
            saved = codes[page, 1, j % 16, 5].clone()
            codes[page, 1, j % 16, 5] = 127
            out, lse = run()
            codes[page, 1, j % 16, 5] = saved
            mine = slice(g, 2 * g)  # the heads of kv head 1
            hit = torch.isnan(out[b, :, mine])
            want = torch.zeros_like(hit)
            want[keepers, :, 5 if what == "v" else slice(None)] = True
            assert torch.equal(hit, want)
            assert torch.equal(torch.isnan(lse[b, :, mine]),
                               keepers[:, None].expand(-1, g) & (what == "k"))
            ok = ~hit
            assert torch.allclose(out[b, :, mine][ok], base[b, :, mine][ok], rtol=2 ** -7, atol=4e-3)
            assert torch.equal(out[b, :, :g], base[b, :, :g]) and torch.equal(out[1 - b], base[1 - b])


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_flags_bad_requests(d, split):
    w = wl.generate(case(d, 2, batch=3, lo=100, hi=200, seed=19))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    q = torch.randn(3, 5, w["hq"], d, device="cuda").to(torch.bfloat16)
    for n, code in (((5, -1, 5), 11), ((5, 6, 5), 11), ((5, 5, 5), 0)):
        out = torch.full_like(q, SENTINEL)
        qb.prefill_sparse(q, torch.tensor(n, dtype=torch.int32, device="cuda"), out, None)
        assert bt.device_error() == code
        dsa.dsa_clear_device_error(bt.ws)
        assert torch.isnan(out[1].float()).all() == (code != 0)
        assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[2].float()).all()


# ---------------------------------------------------------------------------
# a step as a serving loop runs it
# ---------------------------------------------------------------------------

def rotary(hd, axes=3):
    return dsa.make_rope([10000.0 ** (-2 * i / hd) for i in range(hd // 2)],
                         dsa.rope_sections([hd // 2 - 2 * (hd // 8), hd // 8, hd // 8], True))


@pytest.mark.parametrize("d", [64, 128])
def test_step_in_a_loop_and_in_a_graph(d):
    """Rotate the fused projection's q and k, write the new rows, decode -- eagerly step
    by step, and the same steps replayed from one recorded graph on another stream:
    the same cache and outputs, bit for bit, and the oracle's on the final cache."""
    g, hkv, B, steps = 4, 2, 5, 6
    w = wl.generate(case(d, g, batch=B, hkv=hkv, lo=40, hi=120, prompt=(20, 30), W=64, seed=d))
    grow = np.asarray(w["seq_len"]) + steps
    table, pages = wl.make_page_table(grow, True, np.random.default_rng(0))
    w["page_table"], w["num_pages"], w["max_pages"] = table, pages, table.shape[1]
    w["max_kept"] += steps
    gen = torch.Generator().manual_seed(d)
    for name in ("k_pages", "v_pages"):
        w[name] = torch.randn(pages, 16, hkv, d, generator=gen).to(torch.bfloat16)
    qkv = torch.randn(steps, B, (g + 2) * hkv, d, generator=gen).to(torch.bfloat16).cuda()
    pos0 = torch.as_tensor(np.asarray(w["seq_len"]))[:, None].expand(-1, 3).to(torch.int32).cuda()
    rope = rotary(d)

    def fresh():
        qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
        bufs = dict(x=torch.empty_like(qkv[0]), pos=pos0.clone().contiguous(),
                    k=torch.empty(B, hkv, d, dtype=torch.bfloat16, device="cuda"))
        return qb, bufs

    def step(qb, bufs, stream=None):
        bt = qb.batch
        x, hq = bufs["x"], g * hkv
        dsa.dsa_rope_axes(bt.dims, rope, bufs["pos"], x[:, :hq], x[:, hq:hq + hkv], bt.q, bufs["k"],
                          stream)
        # K rotated in its own buffer, V a slice: the write wants one stride, so copy V
        bufs["v"].copy_(x[:, hq + hkv:])
        qb.write(bufs["k"][:, None], bufs["v"][:, None], stream=stream)
        qb.decode_sparse_masked(stream=stream)

    def eager():
        qb, bufs = fresh()
        bufs["v"] = torch.empty_like(bufs["k"])
        outs = []
        for s in range(steps):
            bufs["x"].copy_(qkv[s])
            qb.batch.seq_len += 1
            step(qb, bufs)
            bufs["pos"] += 1
            outs.append((qb.out.clone(), qb.lse.clone()))
        torch.cuda.synchronize()
        assert qb.batch.device_error() == 0
        return qb, outs

    qa, want = eager()
    qb, bufs = fresh()
    bufs["v"] = torch.empty_like(bufs["k"])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(qb, bufs, stream)
    torch.cuda.synchronize()
    for s in range(steps):
        bufs["x"].copy_(qkv[s])
        qb.batch.seq_len += 1
        graph.replay()
        bufs["pos"] += 1
        torch.cuda.synchronize()
        assert torch.equal(qb.out, want[s][0]) and torch.equal(qb.lse, want[s][1])
    for a, b in ((qa.k, qb.k), (qa.v, qb.v), (qa.k_scale, qb.k_scale), (qa.v_scale, qb.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the last step against the oracle on the cache as it is now
    inp = dict(w, seq_len=grow.astype(np.int32), q=qb.batch.q.cpu())
    inp["k_pages"], inp["v_pages"] = dequantised(qb)
    ref, ref_lse = oracle.decode(inp, sparse=True)
    vmax = float(inp["v_pages"].abs().max())
    compare(qb.out.float().cpu(), qb.lse.cpu(), ref, ref_lse, vmax, False)


def test_two_streams_with_their_own_workspaces():
    """Two batches on two streams at once, each its own workspace: the bits of the calls
    made one after the other."""
    qbs = []
    for seed in (1, 2):
        w = wl.generate(case(128, 4, batch=1, hkv=2, lo=4000, hi=4100, prompt=(2000, 2100), W=90, seed=seed))
        qbs.append(QuantBatch.from_batch(DecodeBatch.from_workload(w)))
    want = []
    for qb in qbs:
        qb.decode_dense()
        a = qb.out.clone()
        qb.decode_sparse_masked()
        want.append((a, qb.out.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qbs]
    for _ in range(20):
        outs = []
        for qb, s in zip(qbs, streams):
            with torch.cuda.stream(s):
                a, b = torch.empty_like(qb.out), torch.empty_like(qb.out)
                qb.decode_dense(out=a, stream=s)
                qb.decode_sparse_masked(out=b, stream=s)
                outs.append((a, b))
        torch.cuda.synchronize()
        for got, exp in zip(outs, want):
            assert torch.equal(got[0], exp[0]) and torch.equal(got[1], exp[1])


@pytest.mark.parametrize("n", [4, 20, 70])
def test_chunks_in_a_graph_and_on_two_streams(n):
    """Chunk calls of two batches, captured together and replayed, and issued on two streams
    at once: the bits of eager calls made one after the other."""
    runs = []
    for seed in (1, 2):
        w = wl.generate(case(128, 4, batch=12, hkv=2, lo=90, hi=400, prompt=(30, 60), W=64, seed=seed))
        qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
        gen = torch.Generator().manual_seed(seed)
        q = torch.randn(12, n, w["hq"], 128, generator=gen).to(torch.bfloat16).cuda()
        runs.append((qb, q, torch.as_tensor(chunk_lens(w, n, seed).astype(np.int32)).cuda(),
                     torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device="cuda")))
    for r in runs:
        r[0].prefill_sparse(*r[1:])
    torch.cuda.synchronize()
    want = [(r[3].clone(), r[4].clone()) for r in runs]
    same = lambda: all(torch.equal(r[3], x) and torch.equal(r[4], y) for r, (x, y) in zip(runs, want))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for r in runs:
            r[0].prefill_sparse(*r[1:], stream=stream)
    for _ in range(3):
        for r in runs:
            r[3].fill_(SENTINEL), r[4].fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert same()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        for r, s in zip(runs, streams):
            r[0].prefill_sparse(*r[1:], stream=s)
    torch.cuda.synchronize()
    assert same() and all(r[0].batch.device_error() == 0 for r in runs)


def test_offsets_past_32_bits():
    """The same pages at the far end of a pool whose codes pass 2^32 bytes: the same bits."""
    w = wl.generate(case(128, 4, batch=4, hkv=2, lo=60, hi=200, prompt=(30, 60), W=64, seed=37))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    pages = bt.dims.num_pages
    far = 2 ** 32 // (2 * 16 * 128) + 5
    total = far + pages
    k, v = (torch.empty(total, 2, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((total, 2), float("nan"), device="cuda") for _ in range(2))
    for big, small in ((k, qb.k.view(torch.uint8)), (v, qb.v.view(torch.uint8)), (ks, qb.k_scale),
                       (vs, qb.v_scale)):
        big[far:] = small
    cache = dsa.quant_cache(k, v, ks, vs)
    dims = dsa.dsa_dims.from_buffer_copy(bt.dims)
    dims.num_pages = total
    table = torch.where(bt.page_table >= 0, bt.page_table + far, bt.page_table)
    ws = dsa.alloc_workspace(dims, "cuda")
    out = torch.empty_like(qb.out)
    want = qb.decode_dense()[0].clone()
    dsa.dsa_decode_dense_quant(dims, bt.q, cache, table, bt.seq_len, bt.scale, out, None, ws)
    assert torch.equal(out, want)
    want = qb.decode_sparse_masked()[0].clone()
    dsa.dsa_decode_sparse_masked_quant(dims, bt.q, cache, table, bt.seq_len, bt.prompt_len, bt.window,
                                       bt.keep_mask, bt.scale, out, None, ws)
    assert torch.equal(out, want)
    saved = dsa.dsa_get_prefill_split()
    try:
        for n, split in ((4, 1), (20, 1), (20, 2)):
            dsa.dsa_set_prefill_split(split)
            gen = torch.Generator().manual_seed(n)
            q = torch.randn(4, n, w["hq"], 128, generator=gen).to(torch.bfloat16).cuda()
            ql = torch.full((4,), n, dtype=torch.int32, device="cuda")
            a, b = torch.empty_like(q), torch.empty_like(q)
            qb.prefill_sparse(q, ql, a, None)
            dsa.dsa_prefill_sparse_quant(dims, q, cache, table, bt.seq_len, ql, bt.prompt_len, bt.window,
                                         bt.keep_mask, bt.scale, b, None, ws)
            assert torch.equal(a, b)
    finally:
        dsa.dsa_set_prefill_split(saved)
    rows = torch.randn(4, 3, 2, 128, device="cuda").to(torch.bfloat16)
    dsa.dsa_quant_write(dims, cache, rows, -rows, table, bt.seq_len, None, ws)
    qb.write(rows, -rows)
    start, count = bt.seq_len - 40, torch.full_like(bt.seq_len, 40)
    got = [torch.empty(4, 40, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    dsa.dsa_quant_read(dims, cache, table, bt.seq_len, start, count, got[0], got[1], ws)
    dsa.dsa_quant_read(bt.dims, qb.cache, bt.page_table, bt.seq_len, start, count, got[2], got[3], bt.ws)
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    assert bt.device_error() == 0
    dsa.check_device_error(ws, "far pages")


def test_empty_batches():
    dims = dsa.make_dims(0, 8, 2, 64, 4, 2, 32, 1, 8, "bf16", "bf16")
    real = dsa.make_dims(1, 8, 2, 64, 4, 2, 32, 1, 8, "bf16", "bf16")
    ws = dsa.alloc_workspace(real)
    k, v = (torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.ones(4, 2, device="cuda")
    cache = dsa.quant_cache(k, v, s, s)
    e = lambda *shape, dt=torch.bfloat16: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    i = e(0, dt=torch.int32)
    dsa.dsa_decode_dense_quant(dims, e(0, 8, 64), cache, e(0, 2, dt=torch.int32), i, 0.1, e(0, 8, 64),
                               None, ws)
    dsa.dsa_prefill_sparse_quant(dims, e(0, 3, 8, 64), cache, e(0, 2, dt=torch.int32), i, i, i, i,
                                 e(0, 2, 1, dt=torch.int32), 0.1, e(0, 3, 8, 64), None, ws)
    dsa.dsa_quant_write(dims, cache, e(0, 3, 2, 64), e(0, 3, 2, 64), e(0, 2, dt=torch.int32), i, i, ws)
    dsa.dsa_rope_axes(real, rotary(64), e(0, 3, dt=torch.int32), e(0, 8, 64), e(0, 2, 64), e(0, 8, 64),
                      e(0, 2, 64))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_ref(x, positions, inv_freq, axis, pairing):
    """The rotation in 64 bits; the angle of a far position reduced by whole turns in
    extended arithmetic (Python integers over 2^-80)."""
    d = x.shape[-1]
    ang = np.empty((x.shape[0], d // 2))
    for i in range(d // 2):
        # turns as an exact fraction of the fp64 frequency over 2 pi to 40 digits
        num = int(np.float64(inv_freq[i]).as_integer_ratio()[0])
        den = int(np.float64(inv_freq[i]).as_integer_ratio()[1])
        two_pi = 62831853071795864769252867665590057683943
        for t in range(x.shape[0]):
            p = int(positions[t, axis[i]])
            turns = (num * p * 10 ** 40 * 2 ** 80) // (den * two_pi)
            ang[t, i] = 2 * np.pi * ((turns % 2 ** 80) / 2.0 ** 80)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    x = x.astype(np.float64)
    y = np.empty_like(x)
    lo, hi = (slice(0, d // 2), slice(d // 2, d)) if pairing == "halves" else (slice(0, d, 2),
                                                                               slice(1, d, 2))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def check_rope(got, x, ref, dt):
    """The sine and cosine are off by at most 2^-22 (2^-32 turns, sincospi to 2 units in
    the last place) and the two products and their sum by 2^-23 each, relative to the
    pair's length (<= |x| + |y|); then one rounding to the output."""
    size = np.abs(x.double().cpu().numpy()).max(axis=-1, keepdims=True)
    u = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= u * np.abs(ref) + 2 * size * 2.0 ** -21).all(), err.max()


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("qt,kt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_parity(d, qt, kt, pairing):
    rng = np.random.default_rng(d)
    n, hq, hkv = 11, 6, 3
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    dims = dsa.make_dims(1, hq, hkv, d, 1, 1, 0, 1, 1, qt, kt)
    inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    inv[-3:] = [0.0, 0.0, -0.25]  # a partial embedding, and a pair that turns the other way
    axis = dsa.rope_sections([d // 2 - 2 * (d // 8), d // 8, d // 8], interleaved=True)
    rope = dsa.make_rope(inv, axis, pairing=pairing)
    pos = rng.integers(-50, 5000, (n, 3))
    pos[0], pos[1], pos[2] = 0, 2**31 - 1, -2**31
    q = torch.randn(n, hq, d).to(dts[qt]).cuda()
    k = torch.randn(n, hkv, d).to(dts[kt]).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dp = torch.as_tensor(pos.astype(np.int32)).cuda()
    dsa.dsa_rope_axes(dims, rope, dp, q, k, qo, ko)
    check_rope(qo, q, rope_ref(q.double().cpu().numpy(), pos, inv, axis, pairing), dts[qt])
    check_rope(ko, k, rope_ref(k.double().cpu().numpy(), pos, inv, axis, pairing), dts[kt])
    assert torch.equal(qo[0], q[0]) and torch.equal(ko[0], k[0])  # position 0 turns nothing
    # in place, one of the two alone
    q2 = q.clone()
    dsa.dsa_rope_axes(dims, rope, dp, q2, None, q2, None)
    k2 = k.clone()
    dsa.dsa_rope_axes(dims, rope, dp, None, k2, None, k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_rope_many_tokens_of_a_fused_projection():
    """Enough tokens for several per CTA, not a multiple of it; strided in and out."""
    n, hq, hkv, d = 16 * 152 + 3, 4, 2, 64
    dims = dsa.make_dims(1, hq, hkv, d, 1, 1, 0, 1, 1, "bf16", "bf16")
    inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    axis = dsa.rope_sections([d // 4, d // 4])
    qkv = torch.randn(n, hq + 2 * hkv, d, device="cuda").to(torch.bfloat16)
    keep = qkv.clone()
    pos = torch.randint(0, 100000, (n, 2), device="cuda", dtype=torch.int32)
    dsa.dsa_rope_axes(dims, dsa.make_rope(inv, axis), pos, qkv[:, :hq], qkv[:, hq:hq + hkv],
                      qkv[:, :hq], qkv[:, hq:hq + hkv])
    torch.cuda.synchronize()
    assert torch.equal(qkv[:, hq + hkv:], keep[:, hq + hkv:])  # V untouched
    at = torch.cat([torch.arange(6), torch.arange(n - 6, n)])
    for sl in (slice(0, hq), slice(hq, hq + hkv)):
        x = keep[at.cuda(), sl]
        ref = rope_ref(x.double().cpu().numpy(), pos[at.cuda()].cpu().numpy(), inv, axis, "halves")
        check_rope(qkv[at.cuda(), sl], x, ref, torch.bfloat16)
    # the inverse rotation gives the input back to two roundings
    back = dsa.make_rope([-f for f in inv], axis)
    dsa.dsa_rope_axes(dims, back, pos, qkv[:, :hq], None, qkv[:, :hq], None)
    size = keep[:, :hq].float().abs().amax(-1, keepdim=True)
    assert ((qkv[:, :hq].float() - keep[:, :hq].float()).abs() <= size * 2.0 ** -6).all()
