"""Page assignment from free lists whose count is not one of the list, against the definition (equal),
and on another stream than the current one."""
import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa
from kv_cache_serving_gb300 import workloads as wl
from kv_cache_serving_gb300.session import DecodeBatch, PagePool
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


def step(spare=40):
    w = wl.generate(wl.scaled(wl.WORKLOADS["llamagen-xl"], batch=4), spare_pages=spare)
    bt = DecodeBatch.from_workload(w)
    table = np.pad(w["page_table"], ((0, 0), (0, 2)), constant_values=-1)
    bt.page_table = i32(table)
    bt.dims.max_pages_per_req = table.shape[1]
    bt.ws = dsa.alloc_workspace(bt.dims)
    bt.seq_len.add_(1)
    return w, bt, PagePool(w["num_pages"], table[table >= 0])


def test_outputs_on_another_stream_are_let_go_of_in_its_order():
    """Their memory is not the current stream's to hand out."""
    w, bt, pool = step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pool.assign(bt, stream=s)
    s.synchronize()
    bt.check()
    assert np.array_equal(got[2].cpu().numpy(), w["seq_len"]) and (got[1] >= 0).all()
    at = {t.data_ptr() for t in got}
    del got
    assert not at & {torch.empty(k, dtype=torch.int32, device="cuda").data_ptr() for k in (4, 5, 4, 5)}


def test_assignment_recorded_on_another_stream():
    w, bt, pool = step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dsa.dsa_graph_begin(s)
    start, slot, pos = pool.assign(bt, stream=s)
    g = dsa.dsa_graph_end(s)
    for i in range(3):
        g.launch(s)
        s.synchronize()
        bt.check()
        assert np.array_equal(pos.cpu().numpy(), w["seq_len"] + i) and (slot >= 0).all()
        bt.seq_len.add_(1)
        torch.cuda.synchronize()
    g.close()
