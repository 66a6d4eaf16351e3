"""The calls over shared prefixes refuse bad arguments on the host, before anything reaches a GPU (the
fake pointers are never dereferenced), and the host logic that finds groups and builds such
batches."""
import ctypes

import numpy as np
import pytest
import torch

from kv_cache_serving_gb300 import dsa, session
from kv_cache_serving_gb300 import workloads as wl

BASE = 1 << 20
FAKE, FAR = ctypes.c_void_p(BASE), ctypes.c_void_p(1 << 30)
BAD, UNSUPPORTED, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK


def dims(**over):
    d = dsa.make_dims(2, 8, 2, 128, 10, 4, 96, 3, 50, "bf16", "bf16")
    for name, value in over.items():
        setattr(d, name, value)
    return d


def shared(**over):
    s = dsa.dsa_shared_prefix(1, 40, 24, BASE, BASE)
    for name, value in over.items():
        setattr(s, name, value)
    return s


def call(masked, d=None, s=None, q=FAKE, k=FAKE, v=FAKE, pt=FAKE, L=FAKE, extra=(FAKE, FAKE, FAKE), scale=0.1, out=FAR,
         lse=None, ws=FAKE, null=False):
    lib, D = dsa._load(), ctypes.byref(d or dims())
    S = None if null else ctypes.byref(s or shared())
    if masked:
        return lib.dsa_decode_sparse_masked_shared(D, S, q, k, v, pt, L, *extra, scale, out, lse, ws, None)
    return lib.dsa_decode_dense_shared(D, S, q, k, v, pt, L, scale, out, lse, ws, None)


@pytest.mark.parametrize("masked", [False, True])
def test_refusals(masked):
    at = ctypes.c_void_p
    for kw in (dict(null=True), dict(q=None), dict(k=None), dict(v=None), dict(pt=None), dict(L=None), dict(out=None),
               dict(ws=None), dict(ws=at(BASE + 16)), dict(q=at(BASE + 8)), dict(k=at(BASE + 8)), dict(out=at(BASE + 4)),
               dict(lse=at(BASE + 2)), dict(scale=float("nan")), dict(scale=float("inf")), dict(d=dims(hq=9)),
               dict(s=shared(groups=-1)), dict(s=shared(groups=0)), dict(s=shared(max_prefix=-1)),
               dict(s=shared(max_suffix=-1)), dict(s=shared(max_prefix=65)), dict(s=shared(group_start=None)),
               dict(s=shared(prefix_len=None)),
               dict(out=FAKE), dict(out=at(BASE + 2 * 8 * 128 * 2 - 16)), dict(out=at(BASE - 16))):  # q and out overlap
        assert call(masked, **kw) == BAD, kw
    for kw in (dict(d=dims(q_dtype=dsa.DSA_F32)), dict(d=dims(kv_dtype=dsa.DSA_F32)), dict(d=dims(head_dim=96)),
               dict(d=dims(batch=65536)), dict(d=dims(hkv=65536, hq=65536)),
               dict(d=dims(max_pages_per_req=1 << 25, batch=4096, hkv=64, hq=512),
                    s=shared(max_prefix=1 << 29, groups=4096))):
        kw.setdefault("out", ctypes.c_void_p(1 << 46))
        assert call(masked, **kw) == UNSUPPORTED, kw
    assert call(masked, d=dims(batch=0)) == OK


def test_masked_refusals():
    for i in range(3):
        assert call(True, extra=tuple(None if j == i else FAKE for j in range(3))) == BAD
    assert call(True, d=dims(max_window=1025, mask_words=33)) == UNSUPPORTED


def test_python_checks():
    t = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        dsa.shared_prefix(t, t, 1, 1)  # CPU tensors


def test_shared_groups():
    table = np.array([[1, 2, 3, 4, -1], [1, 2, 3, 9, 8], [1, 2, 7, -1, -1], [5, 6, 7, 8, 9], [5, 6, 7, 8, 1],
                      [5, 4, 3, 2, 1], [0, -1, -1, -1, -1]])
    start, rows = session.shared_groups(table, [64, 80, 48, 80, 80, 80, 3])
    # the third has half of the first two's common rows and more, the sixth only a fourth
    assert start.tolist() == [0, 3, 5, 6, 7] and rows.tolist() == [32, 32, 32, 64, 64, 0, 0]
    # whole pages alone, of the shortest
    start, rows = session.shared_groups(table[:2], [64, 47])
    assert start.tolist() == [0, 2] and rows.tolist() == [32, 32]
    # nothing in common; evicted entries (-1) are no pages
    start, rows = session.shared_groups(np.full((2, 3), -1), [48, 48])
    assert start.tolist() == [0, 1, 2] and rows.tolist() == [0, 0]
    start, rows = session.shared_groups(np.zeros((0, 3), int), [])
    assert start.tolist() == [0] and len(rows) == 0


def test_share_prompts():
    """Requests of a group read the same prompt rows; their own rows and pages are their own."""
    w = wl.generate(wl.scaled(wl.WORKLOADS["llamagen-xl"], batch=6), spare_pages=40)
    sizes = [3, 1, 2]
    s = wl.share_prompts(w, sizes)
    assert s["group_start"].tolist() == [0, 3, 4, 6]
    assert (s["seq_len"] - s["prompt_len"] == w["seq_len"] - w["prompt_len"]).all()

    def rows(t, b, n):
        j = np.arange(n)
        return t[torch.as_tensor(s["page_table"][b, j // 16].astype(np.int64)), torch.as_tensor(j % 16)]
    for g, n in enumerate(sizes):
        first = int(s["group_start"][g])
        P = int(s["prefix_len"][first])
        for b in range(first, first + n):
            assert P == s["prefix_len"][b] == s["prompt_len"][b]
            assert all(torch.equal(rows(s[x], b, P), rows(s[x], first, P)) for x in ("k_pages", "v_pages"))
    own = [set(s["page_table"][b, s["prefix_len"][b] // 16:-(-s["seq_len"][b] // 16)].tolist()) for b in range(6)]
    assert sum(len(o) for o in own) == len(set().union(*own)) and -1 not in set().union(*own)
    start, pre = session.shared_groups(s["page_table"], s["seq_len"])
    assert start.tolist() == [0, 3, 4, 6] and (pre <= s["prefix_len"]).all()
    with pytest.raises(ValueError):
        wl.share_prompts(w, [3, 2])
