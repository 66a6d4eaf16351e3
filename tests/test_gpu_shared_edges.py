"""Decode over shared prefixes: how exact the shared rows' weights are, scales far below one, and
what invalid data does to each request.

Bars of `fine` (relative to sum a |v|, the weighted magnitudes, with a the softmax weights): a weight
is kept as two bf16 numbers, the second of what the first leaves out, so it is off by 2^-8 of
2^-8; a score is a sum of d products in fp32, off by at most d 2^-24 sum |q k| scale, which is the
weight's relative error; 2^x, the subtraction of the reference, the sums of up to some hundreds
of terms and the joining stay below 2^-15.  The output's own rounding is half a step of bf16, 2^-8
of itself."""
import math

import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa
from test_gpu_shared import BF, U, Batch, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


def fine(bt, b):
    """out [hq, d] and its tolerance, in 64 bits."""
    L = int(bt.L[b])
    pages = torch.as_tensor(bt.table[b, :-(-L // 16)], device="cuda")
    k, v = (t[pages].flatten(0, 1)[:L].double() for t in (bt.k, bt.v))
    on = torch.as_tensor(np.stack([bt.rows(b, h) for h in range(bt.hkv)]), device="cuda")
    q = bt.q[b].double().view(bt.hkv, bt.g, bt.d)
    x = torch.einsum("hgd,nhd->hgn", q, k) * bt.scale
    x = x.masked_fill(~on[:, None], -math.inf)
    a = torch.softmax(x, -1)
    off = bt.d * 2.0 ** -24 * abs(bt.scale) * torch.einsum("hgd,nhd->hgn", q.abs(), k.abs())
    out = torch.einsum("hgn,nhd->hgd", a, v)
    # (the weight itself, and its part in the sum that all are divided by)
    size = torch.einsum("hgn,nhd->hgd", a * (off + 2.0 ** -16 + 2.0 ** -15), v.abs())
    size = size + torch.einsum("hgn,hgn->hg", a, off + 2.0 ** -15)[..., None] * out.abs()
    return out.reshape(-1, bt.d), (size * 1.01 + U * (out.abs() + size)).reshape(-1, bt.d)


@pytest.mark.parametrize("S,n", [(2, 3), (3, 40), (16, 8), (130, 9), (700, 5)])
@pytest.mark.parametrize("hkv,g,d,masked", [(2, 4, 128, None), (5, 1, 64, (40, 0.4, 0)), (1, 8, 64, None),
                                            (3, 2, 128, (40, 0.4, 0))])
def test_weights_as_exact_as_those_of_own_rows(S, n, hkv, g, d, masked):
    """Rows of V that cancel each other: what is left of them shows every weight."""
    bt = Batch([n], [S], [i % 3 for i in range(n)], hkv, g, d, masked, seed=S + d)
    sign = torch.where(bt.randn(16, hkv, d) < 0, -1.0, 1.0)  # by slot: copies of a prefix's page are alike
    bt.v.copy_(sign.expand_as(bt.v))
    out, _ = bt.run()
    for b in range(bt.B):
        want, tol = fine(bt, b)
        assert ((out[b].double() - want).abs() <= tol).all(), (b, float(((out[b].double() - want).abs() / tol).max()))
    assert dsa.dsa_get_device_error(bt.ws) == 0


@pytest.mark.parametrize("scale,size", [(0.0, 2.0 ** 60), (2.0 ** -110, 2.0 ** 54), (-2.0 ** -110, 2.0 ** 54),
                                        (2.0 ** -120, 2.0 ** 59)])
def test_scales_far_below_one(scale, size):
    """Scores of up to 2^125 times a scale that brings them down to a few units, or to nothing."""
    bt = Batch([5, 2], [200, 37], [20, 0, 3, 1, 9, 5, 0], 2, 4, 64, seed=2, scale=scale)
    for t in (bt.q, bt.k):
        t.copy_((t.float() * size).to(BF))
    bt.check(*bt.run())
    assert dsa.dsa_get_device_error(bt.ws) == 0


@pytest.mark.parametrize("masked", [None, (40, 0.4, 9)], ids=["dense", "masked"])
@pytest.mark.parametrize("stated", [0, 1, 41])
def test_a_member_states_another_prefix(stated, masked):
    """NaN and BAD_PREFIX, also where what it states is none; its neighbours keep their results, and
    the next call with sound data has all of them."""
    bt = Batch([4, 3], [64, 40], [30] * 7, 2, 4, 128, masked, seed=31)
    bt.shared = dsa.shared_prefix(bt.gs, bt.pre, 64, 100)
    out, lse = bt.run()
    pre = bt.pre.clone()
    bt.pre[5] = stated
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 15
    assert torch.isnan(o2[5].float()).all() and torch.isnan(l2[5]).all()
    good = [0, 1, 2, 3, 4, 6]
    assert torch.equal(out[good], o2[good]) and torch.equal(lse[good], l2[good])
    dsa.dsa_clear_device_error(bt.ws)
    bt.pre.copy_(pre)
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 0 and torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("first,members", [(0, 40), (65, 40), (-1, 40)])
def test_the_first_of_a_group_states_another_prefix(first, members):
    """The group's prefix is what its first request states: members that state another get NaN."""
    bt = Batch([4, 3], [64, 40], [30] * 7, 2, 4, 128, seed=31)
    bt.shared = dsa.shared_prefix(bt.gs, bt.pre, 64, 100)
    out, lse = bt.run()
    bt.pre[4] = first
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) in (14, 15)
    assert torch.equal(out[:4], o2[:4]) and torch.equal(lse[:4], l2[:4])
    assert torch.isnan(o2[5:].float()).all() and torch.isnan(l2[5:]).all()


def test_more_kept_rows_than_the_bound():
    """Under a mask the bound holds per kv head: heads above it get NaN, the others their results."""
    bt = Batch([4, 3], [64, 40], [30] * 7, 4, 2, 128, (40, 0.5, 9), seed=5)
    out, lse = bt.run()
    rest = np.array([[int(bt.rows(b, h).sum()) - int(bt.S[b]) for h in range(bt.hkv)] for b in range(bt.B)])
    bound = int(np.median(rest))
    over = torch.as_tensor(rest > bound, device="cuda").repeat_interleave(bt.g, 1)
    assert over.any() and not over.all()
    o2, l2 = bt.run(dsa.shared_prefix(bt.gs, bt.pre, 64, bound))
    assert dsa.dsa_get_device_error(bt.ws) == 15
    assert torch.isnan(o2[over].float()).all() and torch.isnan(l2[over]).all()
    assert torch.equal(o2[~over], out[~over]) and torch.equal(l2[~over], lse[~over])


@pytest.mark.parametrize("starts", [[1, 1, 5, 8], [0, 1, 5, 7], [0, 9, 8, 8], [0, -1, 5, 8], [0, 1, 5, 10], [3, 2, 1, 0],
                                    [0, 5, 1, 8]])
def test_groups_that_are_no_partition(starts):
    """No prefix is computed then: every request that states one gets NaN, one that states none its
    result."""
    bt = Batch([1, 4, 3], [0, 64, 40], [30] * 8, 2, 4, 128, seed=31)
    out, lse = bt.run()
    gs = bt.gs.clone()
    bt.gs.copy_(i32(starts))
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 14
    assert torch.isnan(o2[1:].float()).all() and torch.isnan(l2[1:]).all()
    assert torch.equal(o2[0], out[0]) and torch.equal(l2[0], lse[0])
    dsa.dsa_clear_device_error(bt.ws)
    bt.gs.copy_(gs)
    o2, l2 = bt.run()
    assert dsa.dsa_get_device_error(bt.ws) == 0 and torch.equal(o2, out) and torch.equal(l2, lse)
