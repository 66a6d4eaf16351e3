"""Head norms with rotary positions, page assignment and row stores on the GPU, against
restatements in 64 bits (whole numbers and copied rows have to be equal).

Bars of the norm (u = 2^-24, fp32's half step, relative; all statistics in fp32): the mean of
d <= 128 squares is a chain of 16 fused steps and 3 shuffled sums, so off by at most 20 u of
itself, the reciprocal root by half of that and 4 u, the products with it and the weight by 2 u:
less than 2^-19 together.  A mean subtracted first is off by 20 u of the largest element, which the
norm scales with the rest: 2^-19 of max |x| / sqrt(var + eps) |w|.  The rotation adds 2^-22 of
sincospi, 2^-24 in products and sums and an angle good to 2^-27 turns (2^-24.3 radians), of the
pair's length: less than 2^-20.  The product's error is relative to the product, not to what a bias
of the other sign leaves of it, so the pair's length is counted as the sum of products and biases.
Together at most 2^-18 of (that + |w| max|x| / sigma), and the output's own rounding: half a step of its type (bf16 2^-8, fp32 2^-24) of itself.
"""
import math

import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


# ---------------------------------------------------------------------------
# head norms
# ---------------------------------------------------------------------------

def norm_ref(x, w, b, eps, kind, positions, inv_freq, pair_axis, pairing):
    """(y, tolerance without the output's rounding), fp64."""
    x = x.double().cpu()
    d = x.shape[-1]
    mu = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    c = x - mu
    root = torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double().cpu()
    bias = torch.zeros(d, dtype=torch.float64) if b is None else b.double().cpu()
    y = c / root * w + bias
    slack = w.abs() * x.abs().amax(-1, keepdim=True) / root if kind == "layer" else torch.zeros_like(y)
    slack = slack + (c / root * w).abs() + bias.abs()
    angle = positions.double().cpu()[:, pair_axis] * torch.tensor(inv_freq, dtype=torch.float64)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    lo, hi = (slice(0, d // 2), slice(d // 2, d)) if pairing == "halves" else (slice(0, d, 2), slice(1, d, 2))
    out, tol = torch.empty_like(y), torch.empty_like(y)
    out[..., lo], out[..., hi] = y[..., lo] * cos - y[..., hi] * sin, y[..., hi] * cos + y[..., lo] * sin
    pair = slack[..., lo] + slack[..., hi]
    tol[..., lo] = tol[..., hi] = pair * 2.0 ** -18
    return out, tol


def norm_case(tokens, hq, hkv, d, qt, kt, wt, kind, per_head, bias, pairing, axes=2, eps=1e-6, seed=0, offset=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dims = dsa.make_dims(1, hq, hkv, d, 1, 1, 0, 1, 1, qt, kt)
    inv = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    axis = [i % axes for i in range(d // 2)]
    rope = dsa.make_rope(inv, axis, pairing=pairing, axes=axes)
    # rows out of a wider projection where q and k have one type
    q = (randn(tokens, hq + 3, d) * torch.exp(randn(tokens, hq + 3, 1)) + offset).to(DT[qt])[:, :hq]
    k = (randn(tokens, hkv + 5, d) * torch.exp(randn(tokens, hkv + 5, 1)) + offset).to(DT[kt])[:, 2:2 + hkv]
    vec = lambda h: (1 + randn(*((h, d) if per_head else (d,)))).to(DT[wt])  # noqa: E731
    w = [vec(hq), vec(hkv)] + ([vec(hq), vec(hkv)] if bias else [None, None])
    norm = dsa.make_qk_norm(kind, eps, *w)
    pos = torch.randint(-5000, 100000, (tokens, axes), generator=gen, device="cuda", dtype=torch.int32)
    return dims, norm, rope, pos, q, k, w, inv, axis


def check_norm(got, x, w, b, eps, kind, pos, inv, axis, pairing):
    ref, tol = norm_ref(x, w, b, eps, kind, pos, inv, axis, pairing)
    tol = tol + HALF_STEP[got.dtype] * (ref.abs() + tol)
    diff = (got.double().cpu() - ref).abs()
    assert torch.isfinite(ref).all() and not (diff > tol).any(), (diff / tol.clamp(min=1e-300)).max()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("tokens,hq,hkv,d,qt,kt,wt,per_head,bias", [
    (1, 1, 1, 64, "bf16", "bf16", "bf16", False, False),
    (3, 8, 2, 128, "bf16", "bf16", "f32", True, True),
    (37, 20, 20, 64, "f32", "f32", "f32", True, False),
    (5, 5, 5, 128, "f32", "bf16", "bf16", False, True),
    (130, 3, 3, 64, "bf16", "f32", "f32", False, True),
    (2501, 6, 3, 128, "bf16", "bf16", "bf16", True, True),   # four tokens per CTA, the last of them alone
    (2435, 7, 7, 64, "f32", "f32", "bf16", False, False),
])
def test_norm(tokens, hq, hkv, d, qt, kt, wt, per_head, bias, kind, pairing):
    dims, norm, rope, pos, q, k, w, inv, axis = norm_case(tokens, hq, hkv, d, qt, kt, wt, kind, per_head, bias,
                                                          pairing, seed=tokens + d)
    qo = torch.full((tokens, hq + 1, d), 7.0, dtype=DT[qt], device="cuda")
    ko = torch.full((tokens, hkv, d), 7.0, dtype=DT[kt], device="cuda")
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, qo[:, :hq], ko)
    check_norm(qo[:, :hq], q, w[0], w[2], 1e-6, kind, pos, inv, axis, pairing)
    check_norm(ko, k, w[1], w[3], 1e-6, kind, pos, inv, axis, pairing)
    assert (qo[:, hq:] == 7).all()  # what lies between the rows stays


def test_norm_in_place_and_halves_of_a_call():
    dims, norm, rope, pos, q, k, w, inv, axis = norm_case(9, 8, 2, 128, "bf16", "bf16", "bf16", "rms", False, False,
                                                          "halves", seed=4)
    qo, ko = torch.empty(9, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(k.contiguous())
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, qo, ko)
    only_q, only_k = torch.empty_like(qo), torch.empty_like(ko)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, None, only_q, None)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, None, k, None, only_k)
    assert torch.equal(qo, only_q) and torch.equal(ko, only_k)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, q, k)  # strided, in place
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_norm_without_weights_or_turning():
    d = 64
    dims, _, _, pos, q, k, _, _, axis = norm_case(11, 4, 4, d, "f32", "f32", "f32", "layer", False, False, "halves")
    rope = dsa.make_rope([0.0] * 32, axis, axes=2)
    qo, ko = torch.empty(11, 4, d, device="cuda"), torch.empty(11, 4, d, device="cuda")
    dsa.dsa_qk_norm_rope(dims, dsa.make_qk_norm("layer", 1e-5), rope, pos, q, k, qo, ko)
    check_norm(qo, q, None, None, 1e-5, "layer", pos, [0.0] * 32, axis, "halves")
    check_norm(ko, k, None, None, 1e-5, "layer", pos, [0.0] * 32, axis, "halves")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("size,eps", [(2.0 ** 120, 1e-6), (2.0 ** 64, 0.0), (2.0 ** -70, 0.0), (2.0 ** -120, 0.0),
                                      (2.0 ** -70, 2.0 ** -140), (2.0 ** -60, 1e-6), (2.0 ** 100, 2.0 ** 100)])
def test_norm_of_very_large_and_small_heads(kind, size, eps):
    """Squares that leave fp32, beside heads of ordinary size in the same warp."""
    dims, _, rope, pos, q, k, w, inv, axis = norm_case(6, 8, 4, 128, "f32", "f32", "f32", kind, False, False, "halves")
    q, k = q.contiguous(), k.contiguous()
    q[:, ::2] *= size / 16
    norm = dsa.make_qk_norm(kind, eps, *w)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, qo, ko)
    check_norm(qo, q, w[0], None, float(np.float32(eps)), kind, pos, inv, axis, "halves")
    check_norm(ko, k, w[1], None, float(np.float32(eps)), kind, pos, inv, axis, "halves")


def test_norm_offset_is_not_cancellation():
    """A mean 1000 times the spread: the squares are taken of what is left."""
    dims, norm, rope, pos, q, k, w, inv, axis = norm_case(6, 8, 4, 128, "f32", "f32", "f32", "layer", True, True,
                                                          "neighbours", offset=1000.0)
    qo, ko = torch.empty(6, 8, 128, device="cuda"), torch.empty(6, 4, 128, device="cuda")
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, qo, ko)
    check_norm(qo, q, w[0], w[2], 1e-6, "layer", pos, inv, axis, "neighbours")


def test_norm_zero_heads_and_nan_stay_apart():
    dims, norm, rope, pos, q, k, w, inv, axis = norm_case(4, 8, 4, 64, "bf16", "bf16", "bf16", "rms", False, False,
                                                          "halves")
    q, k = q.contiguous(), k.contiguous()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q, k, qo, ko)
    q2 = q.clone()
    q2[1, 3], q2[2, 5, 7], q2[0, 6, 9] = 0.0, math.nan, math.inf
    q2o = torch.empty_like(q)
    dsa.dsa_qk_norm_rope(dims, norm, rope, pos, q2, k, q2o, ko)
    assert (q2o[1, 3] == 0).all() and torch.isnan(q2o[2, 5]).all() and torch.isnan(q2o[0, 6]).any()
    same = torch.ones(4, 8, dtype=torch.bool, device="cuda")
    same[1, 3] = same[2, 5] = same[0, 6] = False
    assert torch.equal(q2o[same], qo[same])


# ---------------------------------------------------------------------------
# pages and slots
# ---------------------------------------------------------------------------

def assign_ref(L, n, free, count, table, num_pages, max_tokens):
    """The definition, request by request."""
    table = table.copy()
    B, total = len(L), int(n.sum())
    slot, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    start = np.concatenate([[0], np.cumsum(n)])
    used = 0
    if total <= max_tokens:
        for b in range(B):
            first = -(-(L[b] - n[b]) // 16)
            need = -(-L[b] // 16) - first
            served = need == 0 or used + need <= count
            if not served:
                used = count + 1  # nobody behind it gets pages either
            for i in range(n[b]):
                row = L[b] - n[b] + i
                t = start[b] + i
                pos[t] = row
                if not served:
                    continue
                if row // 16 >= first and row % 16 == 0:
                    pg = free[count - 1 - used - (row // 16 - first)]
                    table[b, row // 16] = pg if 0 <= pg < num_pages else -1
                pg = table[b, row // 16]
                if 0 <= pg < num_pages:
                    slot[t] = pg * 16 + row % 16
            if served:
                used += need
    return table, slot, pos, start


def assign_case(B, lo, hi, nlo, nhi, seed, spare=0, width=None):
    rng = np.random.default_rng(seed)
    L = rng.integers(lo, hi + 1, size=B)
    n = np.minimum(rng.integers(nlo, nhi + 1, size=B), L)
    have = -(-(L - n) // 16)
    need = int((-(-L // 16) - have).sum())
    pool = int(have.sum()) + need + spare + 3
    ids = rng.permutation(pool)
    table = np.full((B, width or (hi + 15) // 16 + 2), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.concatenate([ids[at:at + need + spare], np.full(5, 1 << 29)])
    return L, n, table, free, need + spare, need, pool


def run_assign(L, n, table, free, count, pool, max_tokens, in_place=False, none=False):
    B = len(L)
    dims = dsa.make_dims(B, 1, 1, 64, pool, table.shape[1], 0, 1, 1, "bf16", "bf16")
    ws = dsa.alloc_workspace(dims)
    pt, c = i32(table), i32([count])
    out = c if in_place else i32([-5])
    start = None if none else i32(np.full(B + 1, -9))
    slot = i32(np.full(max_tokens, -9))
    pos = None if none else i32(np.full(max_tokens, -9))
    dsa.dsa_assign_pages(dims, i32(L), None if n is None else i32(n), i32(free), c, out, pt, start, slot, pos, ws)
    code = dsa.dsa_get_device_error(ws)
    get = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
    return code, get(pt), int(out), get(start), get(slot), get(pos)


@pytest.mark.parametrize("B,lo,hi,nlo,nhi,spare,pad", [
    (1, 1, 1, 1, 1, 0, 0), (1, 1, 40, 0, 40, 2, 3), (3, 16, 16, 16, 16, 0, 1), (5, 17, 17, 1, 1, 0, 0),
    (128, 33, 4608, 1, 1, 7, 0), (37, 1, 300, 0, 300, 0, 511), (513, 1, 64, 0, 5, 3, 600), (1100, 1, 90, 0, 33, 1, 7),
    (2, 9000, 9000, 9000, 9000, 0, 0), (600, 1, 20, 0, 0, 4, 20), (4, 1000, 3000, 500, 1500, 0, 513),
])
def test_assign(B, lo, hi, nlo, nhi, spare, pad):
    L, n, table, free, count, need, pool = assign_case(B, lo, hi, nlo, nhi, B + lo)
    count += spare
    free = np.concatenate([free[:need], np.arange(spare) % pool, free[need:]])
    most = int(n.sum()) + pad
    code, pt, left, start, slot, pos = run_assign(L, n, table, free, count, pool, most)
    wt, ws_, wp, wst = assign_ref(L, n, free, count, table, pool, most)
    assert code == 0 and left == count - need
    assert np.array_equal(pt, wt) and np.array_equal(slot, ws_) and np.array_equal(pos, wp) and np.array_equal(start, wst)
    # the count in its own place, and without the optional outputs
    code, pt2, left2, _, slot2, _ = run_assign(L, n, table, free, count, pool, most, in_place=True, none=True)
    assert (code, left2) == (0, left) and np.array_equal(pt2, pt) and np.array_equal(slot2, slot)


def test_assign_default_is_a_decode_step():
    L, n, table, free, count, need, pool = assign_case(40, 1, 100, 1, 1, 3)
    a = run_assign(L, n, table, free, count, pool, 40)
    b = run_assign(L, None, table, free, count, pool, 40)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("short", [1, 2, 17, 10**6])
@pytest.mark.parametrize("B", [6, 700])
def test_assign_serves_whole_requests(short, B):
    """Requests that find too few pages get none; those that need none are served."""
    L, n, table, free, count, need, pool = assign_case(B, 10, 120, 0, 60, B)
    n[-1], L[-1] = 1, 20  # its page is there already
    table[-1, 1] = 0
    need = int((-(-L // 16) - -(-(L - n) // 16)).sum())
    count = max(0, need - short)
    most = int(n.sum()) + 2
    code, pt, left, start, slot, pos = run_assign(L, n, table, free, count, pool, most)
    wt, ws_, wp, wst = assign_ref(L, n, free, count, table, pool, most)
    assert code == 13
    assert np.array_equal(pt, wt) and np.array_equal(slot, ws_) and np.array_equal(pos, wp) and np.array_equal(start, wst)
    fresh = (pt != table).sum()
    assert left == count - fresh


def test_assign_invalid_requests_and_pages():
    L, n, table, free, count, need, pool = assign_case(9, 20, 60, 5, 20, 11)
    # lengths out of range count as no new rows
    L2, n2 = L.copy(), n.copy()
    L2[2], n2[4], n2[6] = 0, -1, L[6] + 1
    code, pt, left, start, slot, pos = run_assign(L2, n2, table, free, count, pool, int(n.sum()))
    n3 = n.copy()
    n3[[2, 4, 6]] = 0
    wt, ws_, wp, wst = assign_ref(L, n3, free, count, table, pool, int(n.sum()))
    assert code in (1, 11)
    assert np.array_equal(pt, wt) and np.array_equal(slot, ws_) and np.array_equal(start, wst)
    # a page id outside the pool, in the free list and in the table
    for bad in (-1, pool, 2**31 - 1):
        free2, table2 = free.copy(), table.copy()
        free2[count - 2] = bad
        b = int(np.flatnonzero((L - n) % 16)[0])
        table2[b, (L - n)[b] // 16] = bad
        code, pt, left, start, slot, pos = run_assign(L, n, table2, free2, count, pool, int(n.sum()))
        wt, ws_, wp, wst = assign_ref(L, n, free2, count, table2, pool, int(n.sum()))
        assert code == 4 and np.array_equal(pt, wt) and np.array_equal(slot, ws_)
    # more new rows than places, and a count that is none: nobody is served
    for cnt, most, want in ((count, int(n.sum()) - 1, 6), (-1, int(n.sum()), 6), (len(free) + 1, int(n.sum()), 6)):
        code, pt, left, start, slot, pos = run_assign(L, n, table, free, cnt, pool, most)
        assert code in (want, 13) and (slot[:0] == -1).all()
        if most < n.sum():
            assert np.array_equal(pt, table) and (slot == -1).all() and left == cnt


def test_assign_empty_batch_and_no_places():
    code, pt, left, start, slot, pos = run_assign(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), int),
                                                  np.arange(3), 3, 10, 5)
    assert code == 0 and left == 3 and start.tolist() == [0] and (slot == -1).all() and (pos == 0).all()
    code, pt, left, *_ = run_assign(np.array([5]), np.array([0]), np.full((1, 2), 3), np.arange(3), 3, 10, 0)
    assert code == 0 and left == 3 and (pt == 3).all()


def test_assign_is_the_way_back_from_eviction():
    """Pages that eviction appends to the free list are handed out again, the last one first."""
    B, W, P, L = 5, 32, 20, np.array([300, 257, 64, 500, 16])
    width, pool = 40, 130
    rng = np.random.default_rng(1)
    ids = rng.permutation(pool)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        k = -(-L[b] // 16)
        table[b, :k] = ids[at:at + k]
        at += k
    dims = dsa.make_dims(B, 1, 1, 64, pool, width, W, 1, 400, "bf16", "bf16")
    ws = dsa.alloc_workspace(dims)
    pt, free, count = i32(table), i32(np.full(pool, -1)), i32([0])
    lens = i32(L)
    dsa.dsa_evict_pages(dims, lens, i32([P] * B), i32([W] * B), pt, free, count, ws)
    evicted, k = pt.clone(), int(count)
    assert k > 10
    n = np.array([16, 3, 40, 0, 1])
    slot = i32(np.zeros(int(n.sum())))
    dsa.dsa_assign_pages(dims, i32(L + n), i32(n), free, count, count, pt, None, slot, None, ws)
    dsa.check_device_error(ws)
    wt, want, _, _ = assign_ref(L + n, n, free.cpu().numpy(), k, evicted.cpu().numpy(), pool, int(n.sum()))
    assert np.array_equal(pt.cpu().numpy(), wt) and np.array_equal(slot.cpu().numpy(), want)
    assert int(count) == k - (wt != evicted.cpu().numpy()).sum()


# ---------------------------------------------------------------------------
# rows at slots
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,hkv,d,dt", [(1, 1, 64, "bf16"), (3, 5, 64, "f32"), (130, 8, 128, "bf16"),
                                             (77, 20, 64, "bf16"), (40, 32, 128, "f32"), (2000, 3, 128, "bf16"),
                                             (9, 9, 128, "bf16")])
def test_write_rows(tokens, hkv, d, dt):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    pages = (tokens + 15) // 16 + 5
    dims = dsa.make_dims(1, hkv, hkv, d, pages, 1, 0, 1, 1, dt, dt)
    ws = dsa.alloc_workspace(dims)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(DT[dt])  # noqa: E731
    kp, vp = randn(pages, 16, hkv, d), randn(pages, 16, hkv, d)
    rows = randn(tokens, 2 * hkv + 1, d)
    k, v = rows[:, :hkv], rows[:, hkv:2 * hkv]
    slot = torch.randperm(pages * 16, generator=gen, device="cuda")[:tokens].to(torch.int32)
    slot[::7] = -1 - slot[::7]  # skipped
    wk, wv = kp.clone(), vp.clone()
    on = slot >= 0
    wk.flatten(0, 1)[slot.long()[on]] = k[on]
    wv.flatten(0, 1)[slot.long()[on]] = v[on]
    k1, v1 = kp.clone(), vp.clone()
    dsa.dsa_write_rows(dims, slot, k, v, k1, v1, ws)
    assert torch.equal(k1, wk) and torch.equal(v1, wv)
    k1, v1 = kp.clone(), vp.clone()  # one of the two, contiguous
    dsa.dsa_write_rows(dims, slot, k.contiguous(), None, k1, None, ws)
    dsa.dsa_write_rows(dims, slot, None, v.contiguous(), None, v1, ws)
    assert torch.equal(k1, wk) and torch.equal(v1, wv)
    assert dsa.dsa_get_device_error(ws) == 0


def test_write_rows_skips_bad_slots():
    dims = dsa.make_dims(1, 2, 2, 64, 4, 1, 0, 1, 1, "f32", "f32")
    ws = dsa.alloc_workspace(dims)
    kp, rows = torch.zeros(4, 16, 2, 64, device="cuda"), torch.ones(4, 2, 64, device="cuda")
    dsa.dsa_write_rows(dims, i32([64, 63, 2**31 - 1, -(2**31)]), rows, None, kp, None, ws)
    assert dsa.dsa_get_device_error(ws) == 4
    assert (kp.flatten(0, 1)[63] == 1).all() and kp.sum() == 128


def test_write_rows_past_32_bits():
    """Slots whose rows lie past 2^32 bytes of the pool."""
    hkv, d, pages = 32, 128, 40000  # 5.2 GB
    dims = dsa.make_dims(1, hkv, hkv, d, pages, 1, 0, 1, 1, "bf16", "bf16")
    ws = dsa.alloc_workspace(dims)
    kp = torch.zeros(pages, 16, hkv, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(3, hkv, d, device="cuda").to(torch.bfloat16)
    slots = [pages * 16 - 1, 16, 33000 * 16 + 5]
    dsa.dsa_write_rows(dims, i32(slots), rows, None, kp, None, ws)
    flat = kp.flatten(0, 1)
    assert all(torch.equal(flat[s], rows[i]) for i, s in enumerate(slots))
    assert int((flat.abs().amax(dim=(1, 2)) > 0).sum()) == 3
