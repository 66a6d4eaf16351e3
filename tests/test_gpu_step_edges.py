"""Page assignment from free lists whose count is not one of the list, against the definition (equal)."""
import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa
from test_gpu_step import assign_case, assign_ref, i32, run_assign

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    torch.cuda.init()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [9, 700])
@pytest.mark.parametrize("more", [1, 1000, 2 ** 30])
def test_a_count_above_the_capacity_is_a_full_list(more, B, in_place):
    """As eviction leaves it when the list was too small: the entries there are go out, the count left
    is one of the list again."""
    L, n, table, free, count, need, pool = assign_case(B, 20, 60, 5, 20, 11)
    free = free[:count]
    for cut in (0, 2):  # all pages that are needed, and two fewer
        lst = free[:count - cut]
        most = int(n.sum()) + 3
        code, pt, left, start, slot, pos = run_assign(L, n, table, lst, len(lst) + more, pool, most, in_place=in_place)
        wt, ws_, wp, wst = assign_ref(L, n, lst, len(lst), table, pool, most)
        assert code == 6 if cut == 0 else code in (6, 13)
        assert np.array_equal(pt, wt) and np.array_equal(slot, ws_) and np.array_equal(pos, wp)
        assert np.array_equal(start, wst) and left == len(lst) - int((wt != table).sum())


@pytest.mark.parametrize("in_place", [False, True])
def test_a_count_below_zero_is_an_empty_list(in_place):
    """Requests whose pages are there are served, the others get none; the count left is 0."""
    L, n, table, free, count, need, pool = assign_case(9, 20, 60, 0, 20, 11)
    n[:3], L[:3] = 1, 20  # their pages are there
    table[:3, 1] = 0
    most = int(n.sum()) + 3
    for bad in (-1, -2 ** 31):
        code, pt, left, start, slot, pos = run_assign(L, n, table, free, bad, pool, most, in_place=in_place)
        wt, ws_, wp, wst = assign_ref(L, n, free, 0, table, pool, most)
        assert code in (6, 13) and left == 0
        assert np.array_equal(pt, wt) and np.array_equal(slot, ws_) and np.array_equal(pos, wp)
        assert np.array_equal(start, wst) and (slot[:3] >= 0).all() and (slot == -1).any()


@pytest.mark.parametrize("most_less", [1, 7, 10 ** 6])
def test_more_rows_than_places_serve_nobody(most_less):
    L, n, table, free, count, need, pool = assign_case(9, 20, 60, 5, 20, 11)
    most = max(0, int(n.sum()) - most_less)
    code, pt, left, start, slot, pos = run_assign(L, n, table, free, count, pool, max(most, 1))
    assert code == 6 and left == count and np.array_equal(pt, table) and (slot == -1).all() and (pos == 0).all()
    assert np.array_equal(start, np.concatenate([[0], np.cumsum(n)]))


def test_eviction_into_a_list_that_is_too_small_and_back():
    """Eviction fills the list and counts on; the next step hands out what the list holds, and the
    one after it counts from there."""
    B, W, P, width, pool = 4, 32, 20, 40, 120
    L = np.array([300, 257, 400, 500])
    ids = np.random.default_rng(2).permutation(pool)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        k = -(-L[b] // 16)
        table[b, :k] = ids[at:at + k]
        at += k
    dims = dsa.make_dims(B, 1, 1, 64, pool, width, W, 1, 400, "bf16", "bf16")
    ws = dsa.alloc_workspace(dims)
    pt, free, count = i32(table), i32(np.full(10, -1)), i32([0])
    dsa.dsa_evict_pages(dims, i32(L), i32([P] * B), i32([W] * B), pt, free, count, ws)
    assert dsa.dsa_get_device_error(ws) == 10 and int(count) > 10
    dsa.dsa_clear_device_error(ws)
    evicted, lst = pt.cpu().numpy(), free.cpu().numpy()
    assert (evicted < 0).sum() - (table < 0).sum() == 10
    n = np.array([16, 3, 40, 1])
    slot = i32(np.zeros(int(n.sum())))
    dsa.dsa_assign_pages(dims, i32(L + n), i32(n), free, count, count, pt, None, slot, None, ws)
    wt, want, _, _ = assign_ref(L + n, n, lst, 10, evicted, pool, int(n.sum()))
    taken = int((wt != evicted).sum())
    assert dsa.dsa_get_device_error(ws) == 6 and taken > 2
    assert np.array_equal(pt.cpu().numpy(), wt) and np.array_equal(slot.cpu().numpy(), want)
    assert int(count) == 10 - taken and (want >= 0).all()
    dsa.dsa_clear_device_error(ws)
    L, now = L + n, pt.cpu().numpy()
    dsa.dsa_assign_pages(dims, i32(L + n), i32(n), free, count, count, pt, None, slot, None, ws)
    wt, want, _, _ = assign_ref(L + n, n, lst, 10 - taken, now, pool, int(n.sum()))
    dsa.check_device_error(ws)
    assert np.array_equal(pt.cpu().numpy(), wt) and np.array_equal(slot.cpu().numpy(), want)
