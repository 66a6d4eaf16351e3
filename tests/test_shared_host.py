"""Host logic of the calls over shared prefixes: which neighbours share, and workspaces."""
import numpy as np
import pytest

from kv_cache_serving_gb300 import dsa, session


def tables(common, own, lens):
    """A table row per request: common[b] lists its pages shared with others, then pages of its own."""
    width, at = max(len(c) for c in common) + own, 10 ** 6
    t = np.full((len(common), width), -1, dtype=np.int64)
    for b, c in enumerate(common):
        t[b, :len(c)] = c
        t[b, len(c):len(c) + own] = np.arange(at, at + own)
        at += own
    return t, lens or [16 * (len(c) + own) for c in common]


def test_a_long_prefix_is_kept_beside_a_request_that_shares_a_page_of_it():
    """One request alone in front of (or behind) eight that have 41 pages in common, the first page in
    common to all."""
    long = list(range(41))
    for common, want in (([[0, 99]] + [long] * 8, [0, 1, 9]), ([long] * 8 + [[0, 99]], [0, 8, 9]),
                         ([[0, 99]] * 2 + [long] * 8, [0, 2, 10]), ([[0, 99]] + [long] * 8 + [[0, 98]] * 3, [0, 1, 9, 12])):
        start, rows = session.shared_groups(*tables(common, 3, None))
        assert start.tolist() == want
        for i, j in zip(want, want[1:]):
            n = 0 if j - i == 1 else 16 * len(common[i])
            if len(common[i]) == 2 and j - i > 1:
                n = 16 * (1 if common[i] != common[i + 1] else 2)
            assert rows[i:j].tolist() == [n] * (j - i)


def saved(table, L, start):
    """Pages read once instead of per request; the groups' common pages."""
    total, common = 0, []
    for i, j in zip(start, start[1:]):
        n = int(min(L[i:j])) // 16
        while n and not ((table[i:j, :n] == table[i, :n]).all() and (table[i, :n] >= 0).all()):
            n -= 1
        total += n * (j - i - 1)
        common.append(n if j - i > 1 else 0)
    return total, common


@pytest.mark.parametrize("seed", range(40))
def test_no_other_cut_saves_more(seed):
    """Against every cut of a small batch whose requests branch off each other anywhere."""
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 9))
    t = np.zeros((B, 6), np.int64)
    t[0] = np.arange(6)
    for b in range(1, B):
        n = int(rng.integers(0, 7))
        t[b] = np.concatenate([t[b - 1, :n], 100 * b + np.arange(6 - n)])
    if seed % 4 == 0:
        t[rng.integers(0, B), rng.integers(0, 6)] = -1
    L = rng.integers(1, 97, size=B)
    start, rows = session.shared_groups(t, L)
    assert start.dtype == rows.dtype == np.int32 and start[0] == 0 and start[-1] == B and (np.diff(start) > 0).all()
    mine, common = saved(t, L, start)
    assert rows.tolist() == np.repeat(np.array(common) * 16, np.diff(start)).tolist()
    assert all(n > 0 for n, k in zip(common, np.diff(start)) if k > 1)
    for bits in range(1 << (B - 1)):
        cut = [0] + [b for b in range(1, B) if bits >> (b - 1) & 1] + [B]
        assert saved(t, L, cut)[0] <= mine


def test_large_batches():
    t = np.repeat(np.arange(40)[None], 3000, 0)
    start, rows = session.shared_groups(t, np.full(3000, 640))
    assert start.tolist() == [0, 3000] and (rows == 640).all()


@pytest.mark.parametrize("batch,hq,hkv,d,pages", [(128, 32, 32, 128, 288), (128, 32, 8, 64, 100), (256, 32, 8, 128, 20),
                                                  (64, 32, 8, 128, 16), (64, 32, 8, 64, 2)])
def test_states_have_a_place_of_their_own_only_where_they_need_one(batch, hq, hkv, d, pages):
    """Split decode keeps a state of d + 2 floats for every 64 rows of a head, 32 at most; four states of
    d + 4 floats fit there, or three more are in the workspace."""
    chunks = min(32, max(1, -(-16 * pages // 64)))
    partials, few = batch * hq * chunks * (d + 2) * 4, chunks * (d + 2) // (d + 4) < 4
    extra = batch * hq * 3 * (d + 4) * 4
    dims = dsa.make_dims(batch, hq, hkv, d, 5000, pages, 96, 3, 16, "bf16", "bf16")
    counts = 4 * batch * (hq + hkv + 1)
    size = dsa.dsa_workspace_size(dims)
    if few:
        assert size >= partials + extra + counts
    else:
        assert partials + counts <= size < partials + counts + min(extra, 1 << 17)
