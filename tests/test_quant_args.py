"""The 8-bit cache and rotary calls refuse bad arguments on the host, before anything
reaches a GPU (the fake pointers are never dereferenced)."""
import ctypes
import math

import pytest
import torch

from kv_cache_serving_gb300 import dsa

BASE = 1 << 20
FAKE = ctypes.c_void_p(BASE)
OFF = ctypes.c_void_p(BASE + 4)


def dims(**over):
    d = dsa.make_dims(2, 8, 2, 128, 10, 4, 96, 3, 50, "bf16", "bf16")
    for name, value in over.items():
        setattr(d, name, value)
    return d


def cache(**over):
    c = dsa.dsa_quant_cache(BASE, BASE, BASE, BASE)
    for name, value in over.items():
        setattr(c, name, value)
    return ctypes.byref(c)


def rope(**over):
    r = dsa.make_rope([0.5] * 64, [0, 1] * 32)
    for name, value in over.items():
        setattr(r, name, value)
    return r


def write(d=None, c=None, max_new=3, k=FAKE, v=FAKE, stride=256, pt=FAKE, L=FAKE, n=None, ws=FAKE):
    return dsa._load().dsa_quant_write(ctypes.byref(d or dims()), c or cache(), max_new, k, v, stride,
                                       pt, L, n, ws, None)


def test_write_refusals():
    bad = dsa.DSA_ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=None), dict(pt=None), dict(L=None), dict(ws=None), dict(max_new=-1),
               dict(stride=255), dict(stride=128), dict(stride=260), dict(k=OFF), dict(v=OFF),
               dict(ws=ctypes.c_void_p(BASE + 16)), dict(c=cache(k_codes=None)),
               dict(c=cache(v_codes=BASE + 8)), dict(c=cache(k_scale=None)), dict(c=cache(v_scale=None)),
               dict(d=dims(kv_dtype=2)), dict(d=dims(batch=-1))):
        assert write(**kw) == bad, kw
    assert dsa._load().dsa_quant_write(ctypes.byref(dims()), None, 3, FAKE, FAKE, 256, FAKE, FAKE, None,
                                       FAKE, None) == bad
    assert write(d=dims(head_dim=96)) == dsa.DSA_ERR_UNSUPPORTED
    assert write(d=dims(num_pages=1 << 28)) == dsa.DSA_ERR_UNSUPPORTED  # rows past 32 bits
    assert write(max_new=0) == dsa.DSA_OK and write(d=dims(batch=0)) == dsa.DSA_OK


def test_read_refusals():
    def read(d=None, c=None, rows=3, pt=FAKE, L=FAKE, s=FAKE, n=FAKE, k=FAKE, v=FAKE, ws=FAKE):
        return dsa._load().dsa_quant_read(ctypes.byref(d or dims()), c or cache(), rows, pt, L, s, n, k, v,
                                          ws, None)
    for kw in (dict(pt=None), dict(L=None), dict(s=None), dict(n=None), dict(ws=None), dict(rows=-1),
               dict(k=OFF), dict(v=OFF), dict(c=cache(k_codes=BASE + 1))):
        assert read(**kw) == dsa.DSA_ERR_INVALID_ARG, kw
    assert read(k=None, v=None) == dsa.DSA_OK and read(rows=0) == dsa.DSA_OK


def attend(name, d=None, c=None, q=FAKE, pt=FAKE, L=FAKE, extra=(FAKE, FAKE, FAKE), scale=0.1, out=FAKE,
           lse=None, ws=FAKE, max_q=3, order=None):
    lib, D, C = dsa._load(), ctypes.byref(d or dims()), c or cache()
    if name == "dense":
        return lib.dsa_decode_dense_quant(D, q, C, pt, L, scale, out, lse, ws, None)
    if name == "list":
        return lib.dsa_decode_sparse_quant(D, q, C, pt, L, extra[0], extra[1], scale, out, lse, ws, None)
    if name == "masked":
        return lib.dsa_decode_sparse_masked_quant(D, q, C, pt, L, *extra, order, scale, out, lse, ws, None)
    return lib.dsa_prefill_sparse_quant(D, max_q, q, C, pt, L, FAKE, *extra, order, scale, out, lse, ws,
                                        None)


@pytest.mark.parametrize("name", ["dense", "list", "masked", "chunk"])
def test_attention_refusals(name):
    for kw in (dict(q=None), dict(pt=None), dict(L=None), dict(out=None), dict(ws=None), dict(q=OFF),
               dict(out=OFF), dict(lse=ctypes.c_void_p(BASE + 2)), dict(ws=ctypes.c_void_p(BASE + 16)),
               dict(scale=math.nan), dict(scale=math.inf), dict(c=cache(k_codes=None)),
               dict(c=cache(v_codes=BASE + 8)), dict(c=cache(v_scale=None)), dict(d=dims(hq=7))):
        assert attend(name, **kw) == dsa.DSA_ERR_INVALID_ARG, kw
    if name != "dense":
        for i in range(2 if name == "list" else 3):
            extra = [FAKE] * 3
            extra[i] = None
            assert attend(name, extra=tuple(extra)) == dsa.DSA_ERR_INVALID_ARG
    assert attend(name, d=dims(head_dim=256)) == dsa.DSA_ERR_UNSUPPORTED
    assert attend(name, d=dims(hq=32)) == dsa.DSA_ERR_UNSUPPORTED      # group 16
    assert attend(name, d=dims(num_pages=1 << 28)) == dsa.DSA_ERR_UNSUPPORTED
    assert attend(name, d=dims(batch=0)) == dsa.DSA_OK


def test_attention_limits():
    wide = dims(max_window=1025, mask_words=33)
    assert attend("masked", d=wide) == dsa.DSA_ERR_UNSUPPORTED
    assert attend("chunk", d=dims(max_window=32769, mask_words=1025)) == dsa.DSA_ERR_UNSUPPORTED
    assert attend("chunk", d=dims(q_dtype=dsa.DSA_F32)) == dsa.DSA_ERR_UNSUPPORTED
    assert attend("chunk", max_q=-1) == dsa.DSA_ERR_INVALID_ARG
    assert attend("chunk", max_q=0) == dsa.DSA_OK


def test_rope_refusals():
    def call(r=None, d=None, n=3, pos=FAKE, q=FAKE, qs=1024, k=FAKE, ks=256, qo=FAKE, qos=1024, ko=FAKE,
             kos=256):
        return dsa._load().dsa_rope_axes(ctypes.byref(d or dims()), ctypes.byref(r or rope()), n, pos, q, qs,
                                         k, ks, qo, qos, ko, kos, None)
    for kw in (dict(n=-1), dict(pos=None), dict(q=None), dict(ko=None), dict(q=OFF), dict(ko=OFF),
               dict(qs=1020), dict(qs=512), dict(kos=128), dict(ks=257), dict(qos=2048),
               dict(r=rope(axes=0)), dict(r=rope(axes=5)), dict(r=rope(axes=1)), dict(r=rope(pairing=2))):
        assert call(**kw) == dsa.DSA_ERR_INVALID_ARG, kw
    for f in (math.nan, math.inf, 7.0):
        r = rope()
        r.inv_freq[63] = f
        assert call(r=r) == dsa.DSA_ERR_INVALID_ARG
    assert dsa._load().dsa_rope_axes(ctypes.byref(dims()), None, 3, FAKE, FAKE, 1024, FAKE, 256, FAKE, 1024,
                                     FAKE, 256, None) == dsa.DSA_ERR_INVALID_ARG
    assert call(n=0) == dsa.DSA_OK
    assert call(q=None, qo=None, k=None, ko=None) == dsa.DSA_OK


def test_binding_checks():
    with pytest.raises(ValueError):
        dsa.make_rope([0.1] * 3, [0] * 4)
    with pytest.raises(ValueError):
        dsa.make_rope([0.1] * 4, [0, 1, 2, 4])
    with pytest.raises(ValueError):
        dsa.make_rope([0.1] * 4, [0] * 4, pairing="odd")
    assert dsa.rope_sections([3, 1, 2]) == [0, 0, 0, 1, 2, 2]
    assert dsa.rope_sections([3, 1, 2], interleaved=True) == [0, 1, 2, 0, 2, 0]
    t = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        dsa.quant_cache(t, t, torch.ones(4, 2), torch.ones(4, 2))  # CUDA tensors wanted
    with pytest.raises(TypeError):
        dsa._cache(dims(), object(), 0)


def test_chunk_refuses_overlapping_q_and_out():
    """[2][3][8][128] bf16: 12 KB each; the same memory, or a byte of it shared, is refused."""
    n = 2 * 3 * 8 * 128 * 2
    for at in (0, 16, n - 16):
        for a, b in ((BASE, BASE + at), (BASE + at, BASE)):
            assert attend("chunk", q=ctypes.c_void_p(a), out=ctypes.c_void_p(b)) == dsa.DSA_ERR_INVALID_ARG
