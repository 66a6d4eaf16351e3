"""The 8-bit cache and the rotary positions at their edges: batches that have grown, softmax
weights far below the largest, tiles with queries that keep nothing or hold NaN, NaN rows of V,
positions of any size.

References are in 64 bits.  Roundings between exact inputs and an output (u = half a step of a
type, relative: bf16 2^-8, fp16 2^-11, fp32 2^-24) are counted beside each comparison.
"""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_serving_gb300 import dsa
from kv_cache_serving_gb300 import workloads as wl
from kv_cache_serving_gb300.session import DecodeBatch, QuantBatch
from test_gpu_quant import TABLE, case, dequantised, split  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


# ---------------------------------------------------------------------------
# batches that have grown, and that share pages
# ---------------------------------------------------------------------------

def same_pool(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in
               ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_from_batch_after_steps(dtype):
    """seq_len advanced on the device, as a serving loop does, before the pages are quantised: the
    pool is that of a batch made with the lengths as they are now."""
    w = wl.generate(case(64, 2, dtype, batch=5, lo=20, hi=90, seed=3), spare_pages=2)
    grow = np.array([0, 1, 5, 16, 40])
    short = dict(w, seq_len=np.maximum(np.asarray(w["seq_len"]) - grow, 1).astype(np.int32))
    bt = DecodeBatch.from_workload(short)
    bt.seq_len += torch.as_tensor(w["seq_len"] - short["seq_len"]).cuda()
    grown = QuantBatch.from_batch(bt)
    assert same_pool(grown, QuantBatch.from_batch(DecodeBatch.from_workload(w)))


def test_from_batch_of_shared_pages():
    """A page that two requests map holds the rows of the longer one, whichever comes last."""
    w = wl.generate(case(64, 2, batch=2, lo=40, hi=40, seed=4))
    alone = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    for order in ((0, 1), (1, 0)):
        shared = dict(w, page_table=np.array(w["page_table"]), seq_len=np.array(w["seq_len"]))
        a, b = order
        shared["page_table"][b, :2] = shared["page_table"][a, :2]
        shared["seq_len"][b] = 24
        qb = QuantBatch.from_batch(DecodeBatch.from_workload(shared))
        at = torch.as_tensor(np.asarray(w["page_table"][a], np.int64)).cuda()
        for x, y in ((qb.k, alone.k), (qb.v, alone.v), (qb.k_scale, alone.k_scale),
                     (qb.v_scale, alone.v_scale)):
            assert torch.equal(x.view(torch.uint8)[at], y.view(torch.uint8)[at])


# ---------------------------------------------------------------------------
# weights far below the largest
# ---------------------------------------------------------------------------

def attend64(w, qb, mode):
    """Decode in 64 bits on the dequantised rows, head by head: out, and the sums that bound what
    roundings do to it -- S = sum w |v| / sum w, the largest w t and sum |code| / sum w of a head
    (t: the V scale of a row's page), B = scale * max_j sum_i |q_i k_ji|, X = the largest |score|."""
    kp, vp = (x.double().numpy() for x in dequantised(qb))
    ts = qb.v_scale.double().cpu().numpy()
    q = qb.batch.q.double().cpu().numpy()
    g, table = w["hq"] // w["hkv"], np.asarray(w["page_table"])
    res = {x: np.zeros(q.shape) for x in ("out", "S", "floor")}
    res.update({x: np.zeros(q.shape[:2]) for x in ("B", "X")})
    for b in range(w["batch"]):
        L = int(w["seq_len"][b])
        for hk in range(w["hkv"]):
            j = np.arange(L) if mode == "dense" else oracle.kept_set(
                L, int(w["prompt_len"][b]), int(w["window"][b]), w["keep_mask"][b, hk])
            pg = table[b, j // 16]
            k, v, t = kp[pg, j % 16, hk], vp[pg, j % 16, hk], ts[pg, hk]
            for h in range(hk * g, hk * g + g):
                x = k @ q[b, h] * qb.batch.scale
                p = np.exp(x - x.max())
                res["out"][b, h] = p @ v / p.sum()
                res["S"][b, h] = p @ np.abs(v) / p.sum()
                res["floor"][b, h] = (p * t).max() * np.abs(v / t[:, None]).sum(0) / p.sum()
                res["B"][b, h] = (np.abs(k) @ np.abs(q[b, h])).max() * qb.batch.scale
                res["X"][b, h] = np.abs(x).max()
    return res


def check_against(w, qb, mode):
    """out against attend64, element by element and relative to what the element is made of.
    A score is off by 2 * 2^-22 B (the halves of q: 11 bits each) and by what fp32 sums of 2 d
    terms lose, 2 d * 2^-23 B, and its exponent by 2^-23 X for each of three roundings; a weight is
    off by as much twice over (numerator and sum), by 2^-22 for 2^x and 2^-22 for its own halves
    or thirds, together 2^-21.  The n weighted rows are added in fp32, n * 2^-23 S at most.  bf16 q: the weights
    round once more, 2^-11 S, or below fp16's normal range by half of its last step, 2^-25 where
    the largest weight (times its page's scale) stands at 2^4 or more; out rounds by 2^-8."""
    out = torch.full_like(qb.out, float("nan"))
    {"dense": qb.decode_dense, "list": qb.decode_sparse, "masked": qb.decode_sparse_masked}[mode](out=out)
    torch.cuda.synchronize()
    assert qb.batch.device_error() == 0
    r = attend64(w, qb, mode)
    d, n = w["head_dim"], int(max(w["seq_len"]))
    score = (2 * 2.0 ** -22 + 2 * d * 2.0 ** -23) * r["B"] + 3 * 2.0 ** -23 * r["X"]
    tol = (2 * np.expm1(score)[..., None] + 2.0 ** -21 + n * 2.0 ** -23) * r["S"]
    if w["dtype"] == "bf16":
        tol = tol + 2.0 ** -11 * r["S"] + 2.0 ** -29 * r["floor"]
        tol = tol + 2.0 ** -8 * (np.abs(r["out"]) + tol)
    else:
        tol = tol + 2.0 ** -24 * np.abs(r["out"])
    err = np.abs(out.double().cpu().numpy() - r["out"])
    bad = ~(err <= tol)
    assert not bad.any(), (mode, (err / tol)[bad].max(), bad.mean())


@pytest.mark.parametrize("lead", [12, 16, 20, 24, 30, 90])
@pytest.mark.parametrize("d,g,dtype", [(64, 1, "f32"), (128, 2, "f32"), (128, 4, "bf16")])
def test_rows_below_a_sink(d, g, dtype, lead):
    """A prompt row whose score leads by 2^lead and whose V is zero: the output is made of
    weights 2^-lead of the largest, which keep their bits."""
    w = wl.generate(case(d, g, dtype, batch=3, lo=150, hi=400, prompt=(100, 140), W=64, seed=lead))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    bt.q[..., 0] = lead * np.log(2) / bt.scale
    w["q"] = bt.q.cpu()
    qb.k_scale.fill_(2.0 ** -5)
    codes = TABLE[qb.k.view(torch.uint8).cpu().numpy()]
    qb.k.copy_(torch.as_tensor(codes / 8).float().cuda().to(torch.float8_e4m3fn))  # scores of about one
    qb.k.view(torch.uint8)[..., 0] = 0
    for b in range(w["batch"]):
        page = int(w["page_table"][b, 0])
        qb.k[page, :, 3] = torch.zeros(d, device="cuda").to(torch.float8_e4m3fn)
        qb.k.view(torch.uint8)[page, :, 3, 0] = int(np.flatnonzero(TABLE == 32.0)[0])
        qb.v.view(torch.uint8)[page, :, 3] = 0
    bt.build_index()
    for mode in ("dense", "list", "masked"):
        check_against(w, qb, mode)


@pytest.mark.parametrize("spread", [12, 30])
@pytest.mark.parametrize("d,g,dtype", [(64, 2, "f32"), (128, 4, "f32"), (128, 4, "bf16"), (64, 1, "bf16")])
def test_scales_far_apart_head_by_head(d, g, dtype, spread):
    """V scales that differ from page to page and head to head by up to 2^60, each head judged by
    its own rows; every fourth page's V is zero whatever its scale."""
    w = wl.generate(case(d, g, dtype, batch=4, lo=200, hi=500, prompt=(150, 180), W=64, seed=spread))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    rng = np.random.default_rng(spread)
    shift = torch.as_tensor(2.0 ** rng.integers(-spread, spread + 1, tuple(qb.v_scale.shape))).float()
    qb.v_scale.copy_(shift)
    qb.v.view(torch.uint8)[::4] = 0
    qb.batch.build_index()
    for mode in ("dense", "list", "masked"):
        check_against(w, qb, mode)


# ---------------------------------------------------------------------------
# chunks: queries that keep nothing, hold NaN, or keep a NaN
# ---------------------------------------------------------------------------

def chunk(qb, q, n):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    ql = torch.full((q.shape[0],), n, dtype=torch.int32, device="cuda")
    qb.prefill_sparse(q, ql, out, lse)
    torch.cuda.synchronize()
    assert qb.batch.device_error() == 0
    return out, lse


def same_bits(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d,g,n", [(128, 1, 5), (128, 4, 5), (128, 1, 40), (64, 2, 5), (64, 4, 20)])
def test_chunk_places_without_a_query_change_nothing(d, g, n, split):
    """A tile that is not full, of whose empty places some keep no row at all under the mask
    (offsets 1 and 2 kept) or every one keeps some (offsets past the chunk kept too, which no
    query of the request reaches): the same bits."""
    w = wl.generate(case(d, g, batch=3, lo=n, hi=n, prompt=(0, 0), W=300, seed=d + n))
    gen = torch.Generator().manual_seed(n)
    q = torch.randn(3, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    w["window"][:] = 300
    got = []
    for far in (False, True):
        bits = np.zeros(w["mask_words"] * 32, np.uint8)
        bits[[0, 1]] = 1
        if far:
            bits[n - 1:300] = 1
        w["keep_mask"][:] = np.packbits(bits, bitorder="little").view(np.uint32)
        got.append(chunk(QuantBatch.from_batch(DecodeBatch.from_workload(w)), q, n))
    assert torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][1]).all()
    assert same_bits(*got)


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d,g,n", [(128, 1, 20), (128, 4, 7), (128, 4, 40), (64, 2, 16), (64, 4, 40)])
def test_chunk_nan_query_leaves_the_others_bits(d, g, n, split):
    w = wl.generate(case(d, g, batch=2, lo=200, hi=260, prompt=(40, 60), W=64, seed=d + n))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    gen = torch.Generator().manual_seed(n)
    q = torch.randn(2, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    want = chunk(qb, q, n)
    x = q.clone()
    x[:, 2, 0, 3] = float("nan")
    got = chunk(qb, x, n)
    assert torch.isnan(got[0][:, 2, 0]).all() and torch.isnan(got[1][:, 2, 0]).all()
    for a, b in zip(want, got):
        b[:, 2, 0] = a[:, 2, 0]
    assert same_bits(want, got)


@pytest.mark.parametrize("split", [0, 1, 2], indirect=True)
@pytest.mark.parametrize("d,g,n", [(128, 1, 20), (128, 4, 7), (128, 4, 40), (64, 2, 16), (64, 4, 40)])
def test_chunk_nan_values_reach_their_element_alone(d, g, n, split):
    """NaN codes of both signs in V rows of the prompt, the window and the chunk: NaN in those
    elements of the queries that keep the row, no sum touched, and elements without a NaN
    within two roundings (fp16 weights, bf16 out) of what they were."""
    w = wl.generate(case(d, g, batch=3, hkv=2, lo=200, hi=260, prompt=(40, 60), W=64, seed=d + n))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    gen = torch.Generator().manual_seed(n)
    q = torch.randn(3, n, w["hq"], d, generator=gen).to(torch.bfloat16).cuda()
    base, lse = chunk(qb, q, n)
    codes = qb.v.view(torch.uint8)
    rng = np.random.default_rng(n)
    want = torch.zeros(base.shape, dtype=torch.bool)
    for b in range(3):
        L, P, W = (int(w[x][b]) for x in ("seq_len", "prompt_len", "window"))
        # request 0: a prompt row; 1: a window row and one of the chunk; 2: many, the last one too
        js = ([5], [L - n - 9, L - n // 2], list(rng.choice(L, 40, replace=False)) + [L - 1])[b]
        for hk in range(2):
            kept = [set(oracle.kept_set(L - n + t + 1, P, W, w["keep_mask"][b, hk])) for t in range(n)]
            for j in js:
                dims = rng.choice(d, 3, replace=False)
                row = codes[int(w["page_table"][b, j // 16]), hk, j % 16]
                row[torch.as_tensor(dims).cuda()] = torch.as_tensor([127, 255, 127], dtype=torch.uint8).cuda()
                for t in range(n):
                    if j in kept[t]:
                        want[b, t, hk * g:hk * g + g, dims] = True
    out, l = chunk(qb, q, n)
    assert torch.equal(torch.isnan(out).cpu(), want)
    assert same_bits([l], [lse])
    # rows that hold a NaN lose nothing but that element: each other element is the same sum
    ok = ~want.cuda()
    assert torch.allclose(out[ok].float(), base[ok].float(), rtol=2 ** -7, atol=4e-3)


@pytest.mark.parametrize("split", [1, 2], indirect=True)
@pytest.mark.parametrize("d,g,n", [(128, 4, 7), (128, 2, 40), (64, 4, 40)])
def test_chunk_nan_values_in_a_graph_and_an_order(d, g, n, split):
    """NaN codes of V with ragged query counts (none for one request), requests handed out in
    another order, without lse, replayed from a graph on another stream: the bits of the plain
    call, and places behind a request's queries left as they were."""
    w = wl.generate(case(d, g, batch=4, hkv=2, lo=150, hi=260, prompt=(40, 60), W=64, seed=d + n))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    bt = qb.batch
    q = torch.randn(4, n, w["hq"], d, device="cuda").to(torch.bfloat16)
    ql = torch.tensor([n, 0, n - 3, 1], dtype=torch.int32, device="cuda")
    codes, rng = qb.v.view(torch.uint8), np.random.default_rng(n)
    for b in range(4):
        L = int(w["seq_len"][b])
        for j in [3] + list(L - 1 - rng.integers(0, 80, 3)):
            codes[int(w["page_table"][b, j // 16]), :, j % 16, int(rng.integers(d))] = 127
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    qb.prefill_sparse(q, ql, out, lse)
    torch.cuda.synchronize()
    assert torch.isnan(out).any() and torch.isfinite(lse).all()
    for b, k in enumerate(ql.tolist()):
        assert (out[b, k:] == 7.0).all() and (lse[b, k:] == 7.0).all()
    got = torch.full_like(q, 7.0)
    order = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        qb.prefill_sparse(q, ql, got, None, stream=stream, request_order=order)
    for _ in range(3):
        got.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        a, b = got.view(torch.int16), out.view(torch.int16)
        assert torch.equal(torch.isnan(got), torch.isnan(out))
        assert torch.equal(a[~torch.isnan(got)], b[~torch.isnan(out)])
    assert bt.device_error() == 0


@pytest.mark.parametrize("split", [0, 1], indirect=True)
@pytest.mark.parametrize("d,n,L", [(128, 8, 2000), (128, 2000, 2000), (64, 8, 2000), (64, 2000, 2000)])
def test_chunk_nan_value_costs_no_more_than_a_few_calls(d, n, L, split):
    """One NaN element in the first V row, which every query keeps, and one in a row that some
    queries keep: no order of magnitude slower than the same call without."""
    w = wl.generate(case(d, 4, batch=4, hkv=4, lo=L, hi=L, prompt=(50, 60), W=300, seed=5))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    q = torch.randn(4, n, w["hq"], d, device="cuda").to(torch.bfloat16)
    out, ql = torch.empty_like(q), torch.full((4,), n, dtype=torch.int32, device="cuda")

    def best():
        times = []
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                qb.prefill_sparse(q, ql, out, None)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) / 3)
        return min(times)

    clean = best()
    codes = qb.v.view(torch.uint8)
    for j in (0, L - 20):
        codes[qb.batch.page_table[:, j // 16].long(), :, j % 16, 3] = 127
    slow = best()
    assert torch.isnan(out.float()).any()
    assert slow <= 6 * clean + 0.02, (slow, clean)  # milliseconds


# ---------------------------------------------------------------------------
# scores of any size
# ---------------------------------------------------------------------------

def huge_case(d, g, dtype, E, L, prompt):
    """Scores of exactly 2^E + 2^s u (log2 units, scale * log2(e) being 1 in fp32), u = 0 in the
    first half of the rows, 1 in the second, 2 in the last quarter of that; all of it exact in fp32."""
    s = max(4, E - 23)
    w = wl.generate(case(d, g, dtype, batch=2, hkv=2, lo=L, hi=L, prompt=(prompt, prompt), W=64, seed=E))
    qb = QuantBatch.from_batch(DecodeBatch.from_workload(w))
    log2e = np.float32(1.4426950408889634)
    near = [np.nextafter(np.float32(np.log(2)), np.float32(x)) for x in (0, 0.5, 1)] + [np.float32(np.log(2))]
    qb.batch.scale = float(next(x for x in near if x * log2e == np.float32(1)))
    codes = np.zeros(tuple(qb.k.shape), np.float32)
    u = np.zeros(L)
    u[L // 2:], u[L - L // 8:] = 1, 2
    for b in range(2):
        page = np.asarray(w["page_table"])[b, np.arange(L) // 16]
        codes[page, :, np.arange(L) % 16, 0] = 16
        codes[page, :, np.arange(L) % 16, 1] = u[:, None]
    qb.k.copy_(torch.as_tensor(codes).cuda().to(torch.float8_e4m3fn))
    qb.k_scale.fill_(1.0)
    qb.v_scale.fill_(1.0)
    qb.v.view(torch.uint8).clamp_(1, 119)  # above zero: an infinite weight would make no NaN
    q = torch.zeros(d, device="cuda")
    q[0], q[1] = 2.0 ** (E - 4), 2.0 ** s
    return w, qb, q, u * 2.0 ** s


def check_huge(w, qb, out, lse, rows, x, E, hk, g, b):
    """out and lse [heads of hk] of one query over `rows`; the roundings are those of any call:
    fp16 weights 2^-11, sums 2^-13, of max |V|, and out's own (bf16 2^-8, fp32 2^-24)."""
    v = dequantised(qb)[1].double().numpy()[np.asarray(w["page_table"])[b, rows // 16], rows % 16, hk]
    p = np.exp2(x[rows] - x[rows].max())
    ref, vmax = p @ v / p.sum(), np.abs(v).max()
    u = 2.0 ** -24 if out.dtype == torch.float32 else 2.0 ** -8
    weights = 0.0 if out.dtype == torch.float32 else 2.0 ** -11
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= u * np.abs(ref) + (weights + 2.0 ** -13) * vmax).all()
    want = (2.0 ** E + x[rows].max() + np.log2(p.sum())) * np.log(2)
    assert (np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -20 * want).all()


@pytest.mark.parametrize("E", [20, 23, 24, 25, 26, 27, 28, 29])
@pytest.mark.parametrize("d,g,dtype", [(128, 4, "bf16"), (64, 1, "bf16"), (128, 2, "f32")])
def test_decode_scores_of_any_size(d, g, dtype, E):
    w, qb, q, x = huge_case(d, g, dtype, E, 640, 500)
    bt = qb.batch
    bt.q.copy_(q.expand_as(bt.q))
    bt.build_index()
    for mode, call in (("dense", qb.decode_dense), ("list", qb.decode_sparse), ("masked", qb.decode_sparse_masked)):
        out, lse = call()
        torch.cuda.synchronize()
        assert bt.device_error() == 0
        for b in range(2):
            for hk in range(2):
                rows = np.arange(640) if mode == "dense" else oracle.kept_set(
                    640, 500, int(w["window"][b]), w["keep_mask"][b, hk])
                check_huge(w, qb, out[b, hk * g:hk * g + g], lse[b, hk * g:hk * g + g], rows, x, E, hk, g, b)


@pytest.mark.parametrize("split", [1, 2], indirect=True)
@pytest.mark.parametrize("E", [20, 24, 25, 26, 27, 28, 29])
@pytest.mark.parametrize("d,g,n", [(128, 4, 5), (128, 1, 40), (64, 2, 12), (64, 4, 40)])
def test_chunk_scores_of_any_size(d, g, n, E, split):
    w, qb, q, x = huge_case(d, g, "bf16", E, 640, 560)
    qs = q.to(torch.bfloat16).expand(2, n, w["hq"], d).contiguous()
    out, lse = chunk(qb, qs, n)
    for b in range(2):
        for hk in range(2):
            for t in (0, n // 2, n - 1):
                rows = oracle.kept_set(640 - n + t + 1, 560, int(w["window"][b]), w["keep_mask"][b, hk])
                check_huge(w, qb, out[b, t, hk * g:hk * g + g], lse[b, t, hk * g:hk * g + g], rows, x, E, hk, g, b)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def _inv_two_pi():
    """1 / (2 pi) over 2^256, rounded down."""
    one = 1 << 320

    def arctan_inv(x):  # arctan(1 / x) over 2^320 (Machin's formula)
        total, term, k, sign = 0, one // x, 1, 1
        while term:
            total += sign * (term // k)
            term //= x * x
            k, sign = k + 2, -sign
        return total

    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    return (one << 256) // (2 * pi)


def rope64(x, positions, inv_freq, axis, pairing):
    """The rotation with its angle reduced to one turn in whole numbers and its sine and cosine
    in 64 bits (of an angle within a quarter turn)."""
    inv, d = _inv_two_pi(), x.shape[-1]
    c, s = (np.empty((x.shape[0], d // 2)) for _ in range(2))
    for i in range(d // 2):
        num, den = float(inv_freq[i]).as_integer_ratio()
        for t in range(x.shape[0]):
            turn = (num * int(positions[t, axis[i]]) * inv // den) % (1 << 256)
            k = (turn + (1 << 253)) >> 254                      # nearest quarter turn
            a = 2 * np.pi * ((turn - (k << 254)) / (1 << 256))
            c[t, i], s[t, i] = ((np.cos(a), np.sin(a)), (-np.sin(a), np.cos(a)), (-np.cos(a), -np.sin(a)),
                                (np.sin(a), -np.cos(a)))[k % 4]
    c, s = c[:, None], s[:, None]
    lo, hi = ((slice(0, d // 2), slice(d // 2, d)) if pairing == "halves" else
              (slice(0, d, 2), slice(1, d, 2)))
    y, size = np.empty(x.shape), np.empty(x.shape)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    size[..., lo] = size[..., hi] = np.abs(x[..., lo]) + np.abs(x[..., hi])
    return y, size


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_angles_to_the_last_bits(d, pairing):
    """Positions from 0 to the ends of their type, frequencies from one turn per position down.
    fp32: the angle is off by 2^-32 turns and by half a step of an fp32 below 1/8, 2^-28 turns,
    together below 2^-25 radians; sine and cosine by 2^-24 (one unit in the last place below 1);
    the two products and their sum by 2^-24 each of what they hold.  Relative to |x| + |y| that
    is 2^-25 + 2^-24 + 2 * 2^-24, below 2^-22."""
    rng = np.random.default_rng(d)
    pos = np.concatenate([np.array([0, 1, -1, 2**31 - 1, -2**31, 2**24 + 1, 2**30 + 12345]),
                          rng.integers(-2**31, 2**31, 30), rng.integers(0, 70000, 30)])[:, None]
    inv = np.concatenate([[2 * np.pi * (1 - 2**-53), 1.0, -1.0, 3.0, 0.7, 1e-3, 6.28, 1e-9, 2.0**-60, np.pi / 2],
                          10000.0 ** (-2 * np.arange(d // 2 - 10) / d)])
    dims = dsa.make_dims(1, 2, 1, d, 1, 1, 0, 1, 1, "f32", "bf16")
    rope = dsa.make_rope(inv, [0] * (d // 2), pairing=pairing)
    q = torch.randn(len(pos), 2, d, device="cuda")
    k = torch.randn(len(pos), 1, d, device="cuda").to(torch.bfloat16)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dsa.dsa_rope_axes(dims, rope, torch.as_tensor(pos.astype(np.int32)).cuda(), q, k, qo, ko)
    for got, x, u in ((qo, q, 0.0), (ko, k, 2.0 ** -8)):
        ref, size = rope64(x.double().cpu().numpy(), pos, inv, [0] * (d // 2), pairing)
        tol = size * 2.0 ** -22
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= tol + u * (np.abs(ref) + tol)).all(), (err / size).max()


@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_leaves_pairs_without_a_frequency(d, pairing, qt):
    """A partial embedding: pairs of inv_freq 0 come out as they went in whatever they hold --
    infinities, NaN, zeros of both signs, the largest and smallest numbers -- and turn nothing
    else; the other pairs are the bits of a call with finite values there."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[qt]
    dims = dsa.make_dims(1, 2, 1, d, 1, 1, 0, 1, 1, qt, qt)
    inv = np.array([10000.0 ** (-2 * i / d) if i < d // 4 else 0.0 for i in range(d // 2)])
    rope = dsa.make_rope(inv, [0] * (d // 2), pairing=pairing)
    pos = torch.tensor([[0], [7], [-3], [2**31 - 1], [100000]], dtype=torch.int32, device="cuda")
    still = np.zeros(d, bool)
    i = np.flatnonzero(inv == 0)
    still[np.concatenate([i, i + d // 2] if pairing == "halves" else [2 * i, 2 * i + 1])] = True
    still = torch.as_tensor(still).cuda()
    q = torch.randn(5, 2, d, device="cuda").to(dt)
    want = torch.empty_like(q)
    dsa.dsa_rope_axes(dims, rope, pos, q, None, want, None)
    special = torch.tensor([float("inf"), -0.0, float("nan"), 1.0, float("-inf"), 0.0, 3e38, 1e-38, -1e-38],
                           device="cuda").to(dt)
    x = q.clone()
    x[..., still] = special[torch.randint(0, 9, x[..., still].shape, device="cuda")]
    got = torch.empty_like(x)
    dsa.dsa_rope_axes(dims, rope, pos, x, None, got, None)
    torch.cuda.synchronize()
    assert same_bits([got[..., ~still]], [want[..., ~still]])
    a, b = got[..., still], x[..., still]
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert same_bits([a.nan_to_num(9.0, posinf=8.0, neginf=-8.0)], [b.nan_to_num(9.0, posinf=8.0, neginf=-8.0)])
