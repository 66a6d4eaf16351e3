"""The 8-bit cache and the rotary positions at their edges: batches that have grown, softmax
weights far below the largest, tiles with queries that keep nothing or hold NaN, NaN rows of V,
positions of any size.

References are in 64 bits.  Roundings between exact inputs and an output (u = half a step of a
type, relative: bf16 2^-8, fp16 2^-11, fp32 2^-24) are counted beside each comparison.
"""
import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa
from kv_cache_serving_gb300 import workloads as wl
from kv_cache_serving_gb300.session import DecodeBatch, QuantBatch
from test_gpu_quant import case

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
