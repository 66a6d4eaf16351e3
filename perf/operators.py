"""Cases of the 8-bit KV cache and its operators: what they compute, on which sizes.

Five operators that a serving step chains on one paged cache:

  rope    rotary positions with several axes (time, height, width) on q and k
  write   new K/V rows quantised into the paged 8-bit cache
  read    rows of the 8-bit cache back as bf16 or fp32
  decode  one query token per request over the 8-bit cache (dense, or the
          prompt and the kept window offsets)
  chunk   several query tokens per request over the 8-bit cache, each over its
          own causal kept set

The cache: codes are e4m3 bytes [num_pages, hkv, 16, head_dim]; one scale, a
power of two, for each (page, kv head) and each of K and V; a row's value is
code * scale.  Here the plain forms are elementary torch operations; with
``own`` set, ``run`` makes the calls of the library instead.  Lengths, masks
and positions belong to the case (``shape_seed``); tensors and the order of the
pages in the pool come from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E_MIN, E_MAX = -40, 40  # exponents a scale may have
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one image token for each request of a mixed serving batch (time, row, column): launch latency counts
        dict(name="rope-step", op="rope", tokens=128, hq=32, hkv=8, d=128, dtype="bf16", axes=3, pairing="halves",
             layout="interleaved", far=1024, shape_seed=1),
        # eight whole 90x90 images with their prompts, straight out of a fused qkv projection
        dict(name="rope-images", op="rope", tokens=65096, hq=32, hkv=8, d=128, dtype="bf16", axes=2,
             pairing="neighbours", layout="blocks", far=100000, shape_seed=2),
        # the step of 32 requests in 24x24 images: one new row each, somewhere inside a page
        dict(name="write-step", op="write", batch=32, hkv=20, d=64, dtype="bf16", seq_lo=121, seq_hi=696,
             new_lo=1, new_hi=1, shape_seed=3),
        # prompts of 64 requests written at once, some behind rows that are there already
        dict(name="write-prompts", op="write", batch=64, hkv=32, d=128, dtype="bf16", seq_lo=256, seq_hi=600,
             new_lo=100, new_hi=256, shape_seed=4),
        # the last window of a few long requests, read back to be looked at in fp32
        dict(name="read-window", op="read", batch=8, hkv=8, d=128, dtype="f32", seq_lo=8000, seq_hi=8250,
             rows_lo=345, rows_hi=360, shape_seed=5),
        # every prompt of a mixed serving batch, back into bf16
        dict(name="read-prompts", op="read", batch=128, hkv=8, d=128, dtype="bf16", seq_lo=512, seq_hi=4608,
             rows_lo=32, rows_hi=512, shape_seed=6),
        # eight long 90x90 images, dense: few units, each cut over many processors
        dict(name="dense-long", op="decode", mode="dense", batch=8, hq=32, hkv=8, d=128, dtype="bf16",
             seq_lo=8000, seq_hi=8250, prompt_lo=64, prompt_hi=64, window=360, shape_seed=7),
        # mixed serving batch, dense: prompts 32..512 and up to 4096 image tokens
        dict(name="dense-mixed", op="decode", mode="dense", batch=128, hq=32, hkv=8, d=128, dtype="bf16",
             seq_lo=33, seq_hi=4608, prompt_lo=32, prompt_hi=512, window=192, shape_seed=8),
        # 24x24 images with fp32 activations: prompt and kept offsets, a few hundred short lists
        dict(name="masked-small", op="decode", mode="masked", batch=32, hq=20, hkv=20, d=64, dtype="f32",
             seq_lo=121, seq_hi=696, prompt_lo=120, prompt_hi=120, window=48, keep=0.2, shape_seed=9),
        # 32x32 images, a mask for each head, every head its own keys
        dict(name="masked-images", op="decode", mode="masked", batch=64, hq=32, hkv=32, d=128, dtype="bf16",
             seq_lo=320, seq_hi=1280, prompt_lo=256, prompt_hi=256, window=96, keep=0.375, shape_seed=10),
        # an image row of 32 tokens at once for each request, under the mask
        dict(name="chunk-row", op="chunk", batch=64, hq=32, hkv=32, d=128, dtype="bf16", seq_lo=320, seq_hi=1280,
             prompt_lo=256, prompt_hi=256, window=96, keep=0.375, new_lo=32, new_hi=32, shape_seed=11),
        # the prompts of a mixed serving batch: every row a query, causal
        dict(name="chunk-prompts", op="chunk", batch=128, hq=32, hkv=8, d=128, dtype="bf16", seq_lo=32, seq_hi=512,
             prompt_lo=512, prompt_hi=512, window=192, keep=0.375, new_lo=512, new_hi=512, shape_seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "decode", "decode", "decode", "chunk", "chunk"])
    g = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 5, 8, 20, 32])
    if hkv * g > 64:
        g = 1
    c = dict(op=op, hkv=hkv, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
             shape_seed=rng.randrange(1 << 30))
    row = hkv * c["d"]
    if op == "rope":
        c.update(hq=hkv * g, axes=rng.choice([1, 2, 3, 4]), pairing=rng.choice(["halves", "neighbours"]),
                 layout=rng.choice(["blocks", "interleaved"]), far=_log(rng, 64, 1 << 24))
        # at most the elements of the largest listed call
        c["tokens"] = _log(rng, 1, min(65096, 150_000_000 // (row * (g + 1))))
        return c
    if op == "write" or op == "read":
        c["batch"] = _log(rng, 1, 128)
        top = max(2, min(4096, 60_000_000 // (row * c["batch"])))
        n = _log(rng, 1, max(1, top // 2))
        lo = max(1, rng.choice([1, n // 2, n]))
        c.update(seq_lo=n, seq_hi=n + _log(rng, 1, top))
        c.update({"new_lo": lo, "new_hi": n} if op == "write" else {"rows_lo": lo, "rows_hi": n})
        return c
    c["batch"] = _log(rng, 1, 128)
    c["hq"] = hkv * g
    c["window"] = rng.choice([0, 1, _log(rng, 2, 400), _log(rng, 2, 1000)])
    c["keep"] = rng.choice([0.1, 0.375, 0.7])
    p = _log(rng, 1, 512)
    c.update(prompt_lo=max(0, p - rng.choice([0, p // 2, p])), prompt_hi=p)
    if op == "decode":
        c["mode"] = rng.choice(["dense", "masked", "list"])
        top = max(4, min(8250, 200_000_000 // (row * c["batch"])))
        hi = _log(rng, 2, top)
        c.update(seq_lo=max(1, rng.choice([1, hi // 2, hi - 16])), seq_hi=hi)
        return c
    c["dtype"] = "bf16"
    n = _log(rng, 2, 512)
    top = max(n + 2, min(2048, 60_000_000 // (row * c["batch"])))
    # at most the score products of the largest listed call
    while c["batch"] > 1 and c["batch"] * c["hq"] * n * (top + n) > 128 * 32 * 300 * 600:
        c["batch"] = (c["batch"] + 1) // 2
    c.update(new_lo=rng.choice([0, n // 2, n]), new_hi=n, seq_lo=n, seq_hi=_log(rng, n + 1, top))
    return c


# ---------------------------------------------------------------------------
# sizes of a case
# ---------------------------------------------------------------------------

def _lengths(case):
    """Per-request lengths and keep masks of a case, on the host."""
    rng = np.random.default_rng(case["shape_seed"])
    B = case["batch"]
    between = lambda x: rng.integers(case[x + "_lo"], case[x + "_hi"] + 1, size=B)  # noqa: E731
    L = between("seq")
    out = dict(L=L)
    if "new_lo" in case:
        out["n"] = np.minimum(between("new"), L)
    if "rows_lo" in case:
        out["n"] = np.minimum(between("rows"), L)
        out["start"] = rng.integers(0, L - out["n"] + 1)
    if "prompt_lo" in case:
        W = case["window"]
        out["P"] = between("prompt")
        out["W"] = rng.integers(W // 2, W + 1, size=B)
        keep = rng.random((B, case["hkv"], max(W, 1))) < case.get("keep", 0.0)
        keep[:, :, :8] = True                                   # the nearest offsets are always kept
        keep &= np.arange(1, max(W, 1) + 1) <= out["W"][:, None, None]
        out["keep"] = keep
    return out


def _words(W):
    return max(1, (W + 31) // 32)


def _bits(keep, words):
    """uint32 words of the keep masks: bit (o-1) keeps window offset o."""
    B, H, W = keep.shape
    k = np.zeros((B, H, words * 32), dtype=np.uint64)
    k[:, :, :W] = keep[:, :, :words * 32]
    k = k.reshape(B, H, words, 32) << np.arange(32, dtype=np.uint64)
    return k.sum(axis=-1).astype(np.uint32)


def _kept_per_query(s, i):
    """Rows that query i of each request keeps, [B, hkv]: prompt, window offsets, itself."""
    L, P, W = s["L"], s["P"], s["W"]
    npr = np.minimum(P, i + 1)
    reach = np.where(i >= npr, np.minimum(i - npr, W), -1)
    cum = np.concatenate([np.zeros(s["keep"].shape[:2] + (1,), np.int64), np.cumsum(s["keep"], axis=2)], axis=2)
    win = np.take_along_axis(cum, np.clip(reach, 0, cum.shape[2] - 1)[:, None, None], axis=2)[:, :, 0]
    return npr[:, None] + np.where(reach[:, None] >= 0, win + 1, 0)


def _max_kept(s):
    return int(np.minimum(s["L"], s["P"] + s["W"] + 1).max())


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["tokens"] * (case["hq"] + hkv) * d
        return {"bytes": 2 * n * e + 4 * case["tokens"] * case["axes"], "flops": 3 * n}
    s = _lengths(case)
    if op == "write":
        n = int(s["n"].sum())
        pages = int(((s["L"] - 1) // PAGE - (s["L"] - s["n"]) // PAGE + 1)[s["n"] > 0].sum())
        return {"bytes": 2 * n * hkv * d * (e + 1) + 8 * pages * hkv, "flops": 4 * n * hkv * d}
    if op == "read":
        n = int(s["n"].sum())
        return {"bytes": 2 * n * hkv * d * (e + 1), "flops": 2 * n * hkv * d}
    if op == "decode":
        rows = int(s["L"].sum()) * hkv if case["mode"] == "dense" else int(_kept_per_query(s, s["L"] - 1).sum())
        qo = case["batch"] * case["hq"] * (2 * d * e + 4)
        return {"bytes": 2 * rows * d + qo, "flops": 4 * rows * (case["hq"] // hkv) * d}
    # chunk: pairs of queries and kept rows; rows that some query of the request keeps
    pairs, rows = 0, 0
    for t in range(int(s["n"].max())):
        live = t < s["n"]
        i = s["L"] - s["n"] + t
        pairs += int(_kept_per_query(s, i)[live].sum())
    for b in range(case["batch"]):
        if s["n"][b] == 0:
            continue
        L, n, P, W = (int(s[k][b]) for k in ("L", "n", "P", "W"))
        j = np.arange(min(P, L), L - n)                          # window rows before the chunk
        hit = np.zeros((hkv, L), dtype=bool)
        hit[:, :min(P, L)] = True
        hit[:, L - n:] = True
        for o in range(1, W + 1):
            near = j[(j + o >= L - n) & (j + o < L)]
            hit[:, near] |= s["keep"][b, :, o - 1][:, None]
        rows += int(hit.sum())
    nq = int(s["n"].sum()) * case["hq"]
    return {"bytes": 2 * rows * d + nq * (2 * d * e + 4), "flops": 4 * pairs * (case["hq"] // hkv) * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _positions(case):
    """[tokens, axes] positions: runs of text (every axis alike), then image tokens (the last two axes run)."""
    rng = np.random.default_rng(case["shape_seed"])
    n, axes = case["tokens"], case["axes"]
    at = rng.integers(0, case["far"], size=1 + n // 8192)
    base = np.repeat(at, 8192)[:n]
    k = np.arange(n) % 8192
    side = 90
    run_of = {axes - 2: k // side, axes - 1: k % side if axes > 1 else k}
    pos = np.stack([base + run_of.get(a, 0) for a in range(axes)], axis=1)
    text = (k < 64)
    pos[text] = (base + k)[text][:, None]
    return pos.astype(np.int32)


def _sections(d, axes):
    """Pairs of a head that each axis turns: the first axis takes what the others leave."""
    each = d // 2 // (axes + 1) if axes > 1 else 0
    return [d // 2 - each * (axes - 1)] + [each] * (axes - 1)


def _pair_axis(case):
    """Axis of each pair: whole blocks, or dealt out in turn until an axis has its share."""
    sec = _sections(case["d"], case["axes"])
    if case["layout"] == "blocks":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    left, out = list(sec), []
    while len(out) < case["d"] // 2:
        for a in range(len(left)):
            if left[a] > 0:
                left[a] -= 1
                out.append(a)
    return out


def _inv_freq(d):
    return [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]


def _values(shape, gen, dtype):
    """Activations: normal, with a spread between heads' rows as projections have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.to(DTYPES[dtype])


def _exponent(amax):
    """Exponent of the scale for a largest magnitude: the smallest e with amax <= 448 * 2^e, within E_MIN..E_MAX."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e in fp32 for whole exponents -126..127, from its bits: pow() need not hit it."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_codes(x, e):
    """e4m3 of x / 2^e, saturated; what is not finite becomes NaN."""
    y = (x.float() * _pow2(-e)).clamp(-448.0, 448.0)
    return torch.where(torch.isfinite(x), y, torch.full_like(y, math.nan)).to(torch.float8_e4m3fn)


def _pool(case, L, gen):
    """A page table in shuffled order and a cache that holds every page's 16 rows."""
    need = (L + PAGE - 1) // PAGE
    pages = int(need.sum()) + 3
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = np.full((len(L), int(need.max())), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    idx = torch.as_tensor(table, device="cuda")
    table = torch.where(idx >= 0, ids[idx.clamp(min=0)], torch.full_like(idx, -1).to(torch.int32))
    st = dict(page_table=table.contiguous())
    for name in ("k", "v"):
        # rows of size about one; pages differ in size as tokens do
        x = torch.randn((pages, case["hkv"], PAGE, case["d"]), generator=gen, device="cuda", dtype=torch.bfloat16)
        size = torch.randint(-2, 3, (pages, 1, 1, 1), generator=gen, device="cuda")
        if name == "v":
            x = (x * _pow2(size)).to(torch.bfloat16)
        e = _exponent(x.abs().amax(dim=(2, 3)).float())
        st[name] = _to_codes(x, e[:, :, None, None])
        st[name + "_scale"] = _pow2(e)
        del x
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d, hkv, dt = case["op"], case["d"], case["hkv"], DTYPES[case["dtype"]]
    if op == "rope":
        n, hq = case["tokens"], case["hq"]
        qkv = _values((n, hq + 2 * hkv, d), gen, case["dtype"])
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv],
                    positions=torch.as_tensor(_positions(case), device="cuda"),
                    q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"),
                    k_out=torch.empty((n, hkv, d), dtype=dt, device="cuda"))
    s = _lengths(case)
    st = _pool(case, s["L"], gen)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")  # noqa: E731
    st.update(case=case, seq_len=dev(s["L"]), pages=st["k"].shape[0])
    B = case["batch"]
    if op == "write":
        n = int(s["n"].max())
        st.update(n=dev(s["n"]), k_new=_values((B, n, hkv, d), gen, case["dtype"]),
                  v_new=_values((B, n, hkv, d), gen, case["dtype"]),
                  touched=int(((s["L"] - 1) // PAGE - (s["L"] - s["n"]) // PAGE + 1)[s["n"] > 0].sum()))
        return st
    if op == "read":
        n = int(s["n"].max())
        st.update(n=dev(s["n"]), start=dev(s["start"]),
                  k_out=torch.zeros((B, n, hkv, d), dtype=dt, device="cuda"),
                  v_out=torch.zeros((B, n, hkv, d), dtype=dt, device="cuda"))
        return st
    W = case["window"]
    st.update(scale=1.0 / math.sqrt(d), prompt_len=dev(s["P"]), window=dev(s["W"]), max_kept=_max_kept(s),
              longest=int(s["L"].max()),
              keep_mask=torch.as_tensor(_bits(s["keep"], _words(W)).view(np.int32), device="cuda"))
    shape = (B, case["hq"], d)
    if op == "chunk":
        shape = (B, max(1, int(s["n"].max())), case["hq"], d)
        st["n"] = dev(s["n"])
    st["q"] = _values(shape, gen, case["dtype"])
    st["out"] = torch.zeros(shape, dtype=dt, device="cuda")
    st["lse"] = torch.zeros(shape[:-1], dtype=torch.float32, device="cuda")
    if op == "decode" and case["mode"] == "list":
        # the kept lists, as a program that keeps them from step to step has them
        keep = _kept(st, (st["seq_len"].long() - 1)[:, None])[:, :, 0]
        idx = torch.sort(keep.int(), dim=-1, descending=True, stable=True).indices[:, :, :st["max_kept"]]
        st["kept_cnt"] = keep.sum(-1).to(torch.int32)
        st["kept_idx"] = torch.zeros((B, hkv, st["max_kept"]), dtype=torch.int32, device="cuda")
        st["kept_idx"][:, :, :idx.shape[2]] = idx.to(torch.int32)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _rope_plain(st):
    case, d = st["case"], st["case"]["d"]
    axis = torch.tensor(_pair_axis(case), device="cuda")
    freq = torch.tensor(_inv_freq(d), dtype=torch.float64, device="cuda")
    angle = st["positions"][:, axis].double() * freq            # far positions: the angle in 64 bits
    turn = 2 * math.pi
    angle = (angle - turn * torch.floor(angle / turn)).float()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    outs = []
    for x in (st["q"], st["k"]):
        x = x.float()
        if case["pairing"] == "halves":
            a, b = x[..., :d // 2], x[..., d // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        outs.append(y.to(DTYPES[case["dtype"]]))
    return {"q": outs[0], "k": outs[1]}


def _write_plain(st):
    n, L = st["n"].long(), st["seq_len"].long()
    B, most = st["k_new"].shape[:2]
    slots = (most + PAGE - 2) // PAGE + 1
    first = (L - n) // PAGE
    row = (first * PAGE)[:, None] + torch.arange(slots * PAGE, device="cuda")       # [B, slots * 16] logical rows
    t = row - (L - n)[:, None]
    new = ((t >= 0) & (t < n[:, None])).view(B, slots, PAGE)
    old = (t < 0).view(B, slots, PAGE)                                                # rows before the new ones
    hit = new.any(-1).flatten()
    pick = torch.sort(hit.int(), descending=True, stable=True).indices[:st["touched"]]
    b, slot = pick // slots, pick % slots
    page = st["page_table"].long()[b, first[b] + slot]
    new, old = new[b, slot][:, None, :, None], old[b, slot][:, None, :, None]
    src = t.view(B, slots, PAGE)[b, slot].clamp(0, most - 1)
    for name in ("k", "v"):
        x = st[name + "_new"][b[:, None], src].permute(0, 2, 1, 3).float()           # [pages, hkv, 16, d]
        size = torch.where(new & torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=(2, 3))
        e = _exponent(size)
        was = st[name][page]
        e_was = torch.frexp(st[name + "_scale"][page])[1] - 1
        e = torch.where(old.flatten(1).any(1)[:, None], torch.maximum(e, e_was), e)
        moved = (was.float() * _pow2(e_was - e)[:, :, None, None]).to(torch.float8_e4m3fn)
        bits = torch.where(new, _to_codes(x, e[:, :, None, None]).view(torch.uint8),
                           torch.where(old, moved.view(torch.uint8), was.view(torch.uint8)))
        st[name].view(torch.uint8)[page] = bits
        st[name + "_scale"][page] = _pow2(e)
    return {x: st[x] for x in ("k", "v", "k_scale", "v_scale")}


def _rows(st, name, b, j):
    """Rows j of requests b for every kv head, [..., hkv, d] in fp32."""
    page = st["page_table"].long()[b, j // PAGE].clamp(min=0)
    x = st[name].view(torch.uint8)[page, :, j % PAGE].view(torch.float8_e4m3fn).float()
    return x * st[name + "_scale"][page][..., None]


def _read_plain(st):
    n, most = st["n"].long(), st["k_out"].shape[1]
    t = torch.arange(most, device="cuda")
    live = (t < n[:, None])
    j = torch.where(live, st["start"].long()[:, None] + t, torch.zeros_like(t))
    b = torch.arange(j.shape[0], device="cuda")[:, None]
    dt = st["k_out"].dtype
    keep = live[:, :, None, None]
    return {x: torch.where(keep, _rows(st, x[0], b, j).to(dt), st[x]) for x in ("k_out", "v_out")}


def _kept(st, i):
    """Whether queries i [B, T] keep row j: [B, hkv, T, longest]."""
    j = torch.arange(st["longest"], device="cuda")
    o = i[:, :, None] - j                                       # [B, T, longest]
    P, W = st["prompt_len"].long()[:, None, None], st["window"].long()[:, None, None]
    bit = (o - 1).clamp(min=0)
    B, hkv, words = st["keep_mask"].shape
    at = (bit // 32).clamp(max=words - 1)[:, None].expand(B, hkv, -1, -1)
    word = torch.gather(st["keep_mask"].long()[:, :, None].expand(-1, -1, at.shape[2], -1), 3, at)
    on = ((word >> (bit % 32)[:, None]) & 1) != 0
    window = (o >= 1) & (o <= W) & (j >= P)
    return ((o >= 0) & ((j < P) | (o == 0)))[:, None] | (window[:, None] & on)


def _attend(q, k, v, keep, scale):
    """q [B, hkv, R, d], k and v [B, hkv, N, d], keep [B, hkv, R or 1, N]: out and the natural logarithm of the sum."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = torch.where(keep, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total
    return out, (m + torch.log(total))[..., 0]


def _decode_plain(st):
    case, B = st["case"], st["case"]["batch"]
    hkv, d = case["hkv"], case["d"]
    L = st["seq_len"].long()
    b = torch.arange(B, device="cuda")[:, None]
    if case["mode"] == "dense":
        j = torch.arange(st["longest"], device="cuda").expand(B, -1)
        live = j < L[:, None]
        j = torch.where(live, j, torch.zeros_like(j))
        k, v = (_rows(st, x, b, j).transpose(1, 2) for x in ("k", "v"))
        keep = live[:, None, None]
    else:
        if case["mode"] == "list":
            idx, count = st["kept_idx"].long(), st["kept_cnt"].long()
        else:
            on = _kept(st, (L - 1)[:, None])[:, :, 0]
            idx = torch.sort(on.int(), dim=-1, descending=True, stable=True).indices[:, :, :st["max_kept"]]
            count = on.sum(-1)
        live = torch.arange(idx.shape[2], device="cuda") < count[:, :, None]
        idx = torch.where(live, idx, torch.zeros_like(idx))
        page = st["page_table"].long()[b[:, :, None], idx // PAGE]
        h = torch.arange(hkv, device="cuda")[None, :, None]
        k, v = (st[x].view(torch.uint8)[page, h, idx % PAGE].view(torch.float8_e4m3fn).float()
                * st[x + "_scale"][page, h][..., None] for x in ("k", "v"))
        keep = live[:, :, None]
    out, lse = _attend(st["q"].float().view(B, hkv, -1, d), k, v, keep, st["scale"])
    return {"out": out.reshape(B, -1, d).to(st["q"].dtype), "lse": lse.reshape(B, -1)}


def _chunk_plain(st):
    case, B = st["case"], st["case"]["batch"]
    hkv, d, g, most = case["hkv"], case["d"], case["hq"] // case["hkv"], st["q"].shape[1]
    L, n = st["seq_len"].long(), st["n"].long()
    b = torch.arange(B, device="cuda")[:, None]
    j = torch.arange(st["longest"], device="cuda").expand(B, -1)
    j = torch.where(j < L[:, None], j, torch.zeros_like(j))
    k, v = (_rows(st, x, b, j).transpose(1, 2) for x in ("k", "v"))
    t = torch.arange(most, device="cuda")
    keep = _kept(st, (L - n)[:, None] + t).repeat_interleave(g, dim=2)               # [B, hkv, T g, longest]
    q = st["q"].float().view(B, most, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, most * g, d)
    out, lse = _attend(q, k, v, keep, st["scale"])
    out = out.view(B, hkv, most, g, d).permute(0, 2, 1, 3, 4).reshape(B, most, -1, d)
    lse = lse.view(B, hkv, most, g).permute(0, 2, 1, 3).reshape(B, most, -1)
    live = (t < n[:, None])[:, :, None]
    return {"out": torch.where(live[..., None], out.to(st["q"].dtype), st["out"]),
            "lse": torch.where(live, lse, st["lse"])}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _handle(st):
    """What a program keeps beside its cache: the dims, the cache's description, the workspace."""
    if "handle" not in st:
        from kv_cache_serving_gb300 import dsa
        c = st["case"]
        hkv, dt = c["hkv"], c["dtype"]
        if c["op"] == "rope":
            dims = dsa.make_dims(1, c["hq"], hkv, c["d"], 1, 1, 0, 1, 1, dt, dt)
            rope = dsa.make_rope(_inv_freq(c["d"]), _pair_axis(c), pairing=c["pairing"])
            st["handle"] = (dsa, dims, rope)
        else:
            W = c.get("window", 0)
            dims = dsa.make_dims(c["batch"], c.get("hq", hkv), hkv, c["d"], st["pages"], st["page_table"].shape[1],
                                 W, _words(W), st.get("max_kept", 1), dt, dt)
            cache = dsa.quant_cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
            st["handle"] = (dsa, dims, cache, dsa.alloc_workspace(dims))
    return st["handle"]


def _run_own(st):
    op = st["case"]["op"]
    if op == "rope":
        dsa, dims, rope = _handle(st)
        dsa.dsa_rope_axes(dims, rope, st["positions"], st["q"], st["k"], st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    dsa, dims, cache, ws = _handle(st)
    if op == "write":
        dsa.dsa_quant_write(dims, cache, st["k_new"], st["v_new"], st["page_table"], st["seq_len"], st["n"], ws)
        return {x: st[x] for x in ("k", "v", "k_scale", "v_scale")}
    if op == "read":
        dsa.dsa_quant_read(dims, cache, st["page_table"], st["seq_len"], st["start"], st["n"], st["k_out"],
                           st["v_out"], ws)
        return {"k_out": st["k_out"], "v_out": st["v_out"]}
    if op == "chunk":
        dsa.dsa_prefill_sparse_quant(dims, st["q"], cache, st["page_table"], st["seq_len"], st["n"], st["prompt_len"],
                                     st["window"], st["keep_mask"], st["scale"], st["out"], st["lse"], ws)
    elif st["case"]["mode"] == "dense":
        dsa.dsa_decode_dense_quant(dims, st["q"], cache, st["page_table"], st["seq_len"], st["scale"], st["out"],
                                   st["lse"], ws)
    elif st["case"]["mode"] == "list":
        dsa.dsa_decode_sparse_quant(dims, st["q"], cache, st["page_table"], st["seq_len"], st["kept_idx"],
                                    st["kept_cnt"], st["scale"], st["out"], st["lse"], ws)
    else:
        dsa.dsa_decode_sparse_masked_quant(dims, st["q"], cache, st["page_table"], st["seq_len"], st["prompt_len"],
                                           st["window"], st["keep_mask"], st["scale"], st["out"], st["lse"], ws)
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "write": _write_plain, "read": _read_plain, "decode": _decode_plain,
            "chunk": _chunk_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e in fp64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _code_values(x):
    """The value of each e4m3 code, from its sign, exponent and mantissa."""
    u = x.view(torch.uint8).long()
    sign, ex, man = 1 - 2 * (u >> 7), (u >> 3) & 15, u & 7
    val = torch.where(ex > 0, (8 + man) * _two_to(ex - 10), man * 2.0 ** -9)
    return torch.where((u & 127) == 127, torch.full_like(val, math.nan), sign * val)


def _nearest_code(x):
    """The e4m3 value nearest to x (fp64), ties to the even mantissa, saturated at 448."""
    a = x.abs().clamp(max=448.0)
    step = _two_to((torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _exact_rope(st):
    case, d = st["case"], st["case"]["d"]
    axis = _pair_axis(case)
    out = {}
    angle = torch.stack([st["positions"][:, a].double() * 10000.0 ** (-2.0 * i / d) for i, a in enumerate(axis)], dim=1)
    for name in ("q", "k"):
        x = st[name].double()
        y = torch.empty_like(x)
        lo = slice(0, d // 2) if case["pairing"] == "halves" else slice(0, d, 2)
        hi = slice(d // 2, d) if case["pairing"] == "halves" else slice(1, d, 2)
        z = torch.polar(torch.ones_like(angle), angle)[:, None] * torch.complex(x[..., lo], x[..., hi])
        y[..., lo], y[..., hi] = z.real, z.imag
        out[name] = y
    return out


def _exact_write(st):
    L, n, table = st["seq_len"].tolist(), st["n"].tolist(), st["page_table"].tolist()
    out = {}
    for name in ("k", "v"):
        codes, scale = _code_values(st[name]), st[name + "_scale"].double()
        for b in range(len(L)):
            first = L[b] - n[b]
            for p in range(first // PAGE, (L[b] - 1) // PAGE + 1) if n[b] else ():
                lo, hi = max(first, p * PAGE), min(L[b], (p + 1) * PAGE)
                x = st[name + "_new"][b, lo - first:hi - first].double().transpose(0, 1)      # [hkv, rows, d]
                page, at = table[b][p], lo - p * PAGE
                fine = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=(1, 2))
                m, e = torch.frexp(fine / 448.0)
                e = torch.where(fine > 0, e - (m == 0.5).int(), torch.full_like(e, E_MIN))
                want = _two_to(e.clamp(E_MIN, E_MAX))
                if at > 0:
                    want = torch.maximum(want, scale[page])
                    codes[page, :, :at] = _nearest_code(codes[page, :, :at] * (scale[page] / want)[:, None, None])
                codes[page, :, at:at + hi - lo] = _nearest_code(x / want[:, None, None])
                scale[page] = want
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_read(st):
    out = {"k_out": st["k_out"].double(), "v_out": st["v_out"].double()}
    for b, (s, n) in enumerate(zip(st["start"].tolist(), st["n"].tolist())):
        k, v = _exact_kv(st, b, s + n)
        out["k_out"][b, :n], out["v_out"][b, :n] = k[:, s:].transpose(0, 1), v[:, s:].transpose(0, 1)
    return out


def _exact_kv(st, b, L):
    """The first L rows of request b, [hkv, L, d] each of K and V."""
    ids = st["page_table"][b, :(L + PAGE - 1) // PAGE].long()
    found = []
    for name in ("k", "v"):
        x = _code_values(st[name][ids]) * st[name + "_scale"][ids].double()[:, :, None, None]
        found.append(x.transpose(0, 1).flatten(1, 2)[:, :L])
    return found


def _exact_attend(st):
    case = st["case"]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    s = _lengths(case)
    chunk = case["op"] == "chunk"
    q, out, lse = st["q"].double(), st["out"].double(), st["lse"].double()
    if not chunk:
        q, out, lse = q[:, None], out[:, None], lse[:, None]
    keep_all = torch.as_tensor(s["keep"], device="cuda")
    for b in range(case["batch"]):
        L, P, W = int(s["L"][b]), int(s["P"][b]), int(s["W"][b])
        n = int(s["n"][b]) if chunk else 1
        if n == 0:
            continue
        k, v = _exact_kv(st, b, L)
        i = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        o = i - j
        if not chunk and case["mode"] == "dense":
            keep = (o >= 0)[None].expand(hkv, -1, -1)
        else:
            near = keep_all[b][:, (o - 1).clamp(0, keep_all.shape[2] - 1)] & ((o >= 1) & (o <= W))
            keep = (o >= 0) & ((j < P) | (o == 0) | near)
        qb = q[b, :n].view(n, hkv, g, -1).permute(1, 2, 0, 3)                        # [hkv, g, n, d]
        x = (qb @ k[:, None].transpose(-1, -2)) / math.sqrt(case["d"])
        x = x.masked_fill(~keep[:, None], -math.inf)
        lse[b, :n] = torch.logsumexp(x, dim=-1).permute(2, 0, 1).reshape(n, -1)
        out[b, :n] = (torch.softmax(x, dim=-1) @ v[:, None]).permute(2, 0, 1, 3).reshape(n, hkv * g, -1)
    return {"out": out if chunk else out[:, 0], "lse": lse if chunk else lse[:, 0]}


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "decode": _exact_attend,
                "chunk": _exact_attend}[case["op"]](st)
