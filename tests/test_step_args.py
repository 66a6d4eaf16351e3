"""Head norms, page assignment and row stores refuse bad arguments on the host, before anything
reaches a GPU (the fake pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from kv_cache_serving_gb300 import dsa

BASE = 1 << 20
FAKE = ctypes.c_void_p(BASE)
OFF = ctypes.c_void_p(BASE + 4)
BAD, UNSUPPORTED, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK


def dims(**over):
    d = dsa.make_dims(2, 8, 2, 128, 10, 4, 96, 3, 50, "bf16", "bf16")
    for name, value in over.items():
        setattr(d, name, value)
    return d


def norm(**over):
    n = dsa.dsa_qk_norm(dsa.NORM_RMS, 0, dsa.DSA_BF16, 1e-6, BASE, BASE, None, None)
    for name, value in over.items():
        setattr(n, name, value)
    return n


def rope(**over):
    r = dsa.make_rope([0.5] * 64, [0, 1] * 32)
    for name, value in over.items():
        setattr(r, name, value)
    return r


def turn(d=None, n=None, r=None, tokens=3, pos=FAKE, q=FAKE, qs=1024, k=FAKE, ks=256, qo=FAKE, qos=1024, ko=FAKE,
         kos=256, null_norm=False):
    return dsa._load().dsa_qk_norm_rope(
        ctypes.byref(d or dims()), None if null_norm else ctypes.byref(n or norm()), ctypes.byref(r or rope()), tokens,
        pos, q, qs, k, ks, qo, qos, ko, kos, None)


def test_norm_refusals():
    for kw in (dict(null_norm=True), dict(n=norm(kind=2)), dict(n=norm(kind=-1)), dict(n=norm(weight_dtype=2)),
               dict(n=norm(eps=-1e-6)), dict(n=norm(eps=float("nan"))), dict(n=norm(eps=float("inf"))),
               dict(n=norm(q_weight=BASE + 8)), dict(n=norm(k_weight=BASE + 2)), dict(n=norm(q_bias=BASE + 4)),
               dict(n=norm(k_bias=BASE + 4)), dict(r=rope(axes=5)), dict(r=rope(pairing=3)), dict(tokens=-1),
               dict(pos=None), dict(q=None), dict(ko=None), dict(q=OFF), dict(qs=1023), dict(ks=255), dict(qos=1020),
               dict(q=FAKE, qo=FAKE, qs=1024, qos=2048), dict(d=dims(batch=-1))):
        assert turn(**kw) == BAD, kw
    assert turn(d=dims(head_dim=96)) == UNSUPPORTED
    assert turn(tokens=0) == OK and turn(q=None, qo=None, k=None, ko=None) == OK


def assign(d=None, L=FAKE, n=None, free=FAKE, cap=5, count=FAKE, out=FAKE, pt=FAKE, most=8, start=None, slot=FAKE,
           pos=None, ws=FAKE):
    return dsa._load().dsa_assign_pages(ctypes.byref(d or dims()), L, n, free, cap, count, out, pt, most, start, slot,
                                        pos, ws, None)


def test_assign_refusals():
    for kw in (dict(L=None), dict(free=None), dict(cap=-1), dict(count=None), dict(out=None), dict(pt=None),
               dict(most=-1), dict(slot=None), dict(ws=None), dict(ws=ctypes.c_void_p(BASE + 16)),
               dict(d=dims(hq=9))):
        assert assign(**kw) == BAD, kw
    assert assign(d=dims(page_size=32)) == UNSUPPORTED
    assert assign(d=dims(num_pages=1 << 27)) == UNSUPPORTED  # slots past int32


def write(d=None, tokens=3, slot=FAKE, k=FAKE, ks=256, v=FAKE, vs=256, kp=FAKE, vp=FAKE, ws=FAKE):
    return dsa._load().dsa_write_rows(ctypes.byref(d or dims()), tokens, slot, k, ks, v, vs, kp, vp, ws, None)


def test_write_refusals():
    for kw in (dict(tokens=-1), dict(slot=None), dict(slot=ctypes.c_void_p(BASE + 2)), dict(k=None), dict(vp=None),
               dict(k=OFF), dict(vp=OFF), dict(ks=255), dict(vs=260), dict(ks=128), dict(ws=None),
               dict(ws=ctypes.c_void_p(BASE + 8)), dict(d=dims(kv_dtype=5))):
        assert write(**kw) == BAD, kw
    assert write(d=dims(head_dim=80)) == UNSUPPORTED
    wide = dims(hq=1 << 20, hkv=1 << 20)  # more 2 KB pieces than a launch takes
    assert write(d=wide, tokens=1 << 20, ks=1 << 27, vs=1 << 27) == UNSUPPORTED
    assert write(tokens=0) == OK and write(k=None, kp=None, v=None, vp=None) == OK


def test_python_checks():
    """The binding names what is wrong before the C call (CPU tensors never get that far)."""
    with pytest.raises(ValueError):
        dsa.make_qk_norm("batch", 1e-6)
    with pytest.raises(TypeError):
        dsa.make_qk_norm("rms", 1e-6, q_weight=torch.ones(128))
    assert dsa.make_qk_norm("layer", 0.0).kind == dsa.NORM_LAYER
    r = dsa.make_rope([0.5] * 32, [0] * 32)
    x = torch.zeros(3, 1, dtype=torch.int32)
    with pytest.raises(ValueError):  # 32 pairs for a head of 128
        dsa.dsa_qk_norm_rope(dims(), dsa.make_qk_norm("rms", 0.0), r, x, None, None, None, None)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(dims(), dsa.make_qk_norm("rms", 0.0), r, x[:, 0], None, None, None, None)
