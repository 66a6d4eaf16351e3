"""Tensors that the session classes make for a call belong to the stream the call is launched on (no
GPU: the library's calls, streams and allocations are stood in for)."""
import contextlib

import pytest
import torch

from kv_cache_serving_gb300 import dsa, session
from kv_cache_serving_gb300 import workloads as wl


@pytest.fixture
def world(monkeypatch):
    """(batch, stream, made): made lists the stream that each tensor was made on, and the call."""
    w = wl.generate(wl.scaled(wl.WORKLOADS["llamagen-xl"], batch=2))
    bt = session.DecodeBatch.from_workload(w, device="cpu")
    made, now, state = [], [None], {"recording": False}

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s if s is not None else now[0]
        yield
        now[0] = before
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0] == "s" and state["recording"])
    for name in ("empty", "full", "zeros", "empty_like"):
        def make(*a, real=getattr(torch, name), **k):
            made.append(now[0])
            return real(*a, **k)
        monkeypatch.setattr(torch, name, make)
    for name in ("dsa_assign_pages", "dsa_evict_pages", "dsa_attention_mass", "dsa_decode_dense_shared",
                 "dsa_decode_sparse_masked_shared"):
        monkeypatch.setattr(dsa, name, lambda *a: made.append(("call", a[-1])))
    pool = object.__new__(session.PagePool)
    pool.free, pool.count = torch.zeros(4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    made.clear()
    return bt, pool, made, state


CALLS = {"assign": lambda bt, pool, s: pool.assign(bt, stream=s), "evict": lambda bt, pool, s: bt.evict_pages(stream=s),
         "mass": lambda bt, pool, s: bt.attention_mass(stream=s),
         "dense": lambda bt, pool, s: bt.decode_dense_shared(None, stream=s),
         "masked": lambda bt, pool, s: bt.decode_sparse_masked_shared(None, stream=s)}


@pytest.mark.parametrize("what", CALLS)
@pytest.mark.parametrize("s", [None, "s"])
def test_outputs_are_made_on_the_stream_of_the_call(world, what, s):
    bt, pool, made, state = world
    CALLS[what](bt, pool, s)
    assert len(made) > 1 and made[-1] == ("call", s) and all(m == s for m in made[:-1])


@pytest.mark.parametrize("what", CALLS)
def test_a_recording_stream_allocates_nothing(world, what):
    bt, pool, made, state = world
    state["recording"] = True
    CALLS[what](bt, pool, "s")
    assert len(made) > 1 and made[-1] == ("call", "s") and all(m is None for m in made[:-1])


def test_the_context_hands_on_what_is_raised(world):
    for s in (None, "s"):
        with pytest.raises(ValueError):
            with session._made_on(s):
                raise ValueError
