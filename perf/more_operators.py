"""Cases of the operators around a paged K/V cache that requests share and fill by themselves: what
they compute, on which sizes.

Four operators of one serving step for requests that continue the same prompt (many images of one
prompt, many answers behind one instruction):

  pages   page tables and row slots built on the GPU: the new rows of every request get pages from
          the free list
  norm    the query and key heads of new tokens normed, each head for itself (root mean square, or
          mean and variance), and turned to their positions in the same pass
  rows    new K/V rows stored at their slots
  shared  one query token per request over the cache, the prefix that a group of requests shares
          attended once for all of them, the rest row by row (dense, or the prompt and the kept
          window offsets)

K and V pages are [num_pages, 16, hkv, head_dim]; row j of request b lies in page
page_table[b][j / 16] at slot j % 16.  Here the plain forms are elementary torch operations; with
``own`` set, ``run`` makes the calls of the library instead.  Lengths, masks and positions belong to
the case (``shape_seed``); tensors and the order of the pages in the pool come from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one image token for each request of a mixed serving batch (time, row, column): latency counts
        dict(name="norm-step", op="norm", tokens=128, hq=32, hkv=8, d=128, dtype="bf16", kind="rms", per_head=False,
             axes=3, pairing="halves", far=1024, shape_seed=21),
        # eight whole 90x90 images with their prompts, out of a fused qkv projection; a norm with
        # mean, weight and bias of every head's own
        dict(name="norm-images", op="norm", tokens=65096, hq=32, hkv=8, d=128, dtype="bf16", kind="layer",
             per_head=True, axes=2, pairing="neighbours", far=100000, shape_seed=22),
        # the prompts of 32 requests in fp32, every head its own keys
        dict(name="norm-prompts-f32", op="norm", tokens=3845, hq=20, hkv=20, d=64, dtype="f32", kind="rms",
             per_head=False, axes=1, pairing="halves", far=700, shape_seed=23),
        # one new row for each request of a mixed serving batch: most go on in their last page
        dict(name="pages-step", op="pages", batch=128, seq_lo=33, seq_hi=4608, new_lo=1, new_hi=1, pad=0, shape_seed=24),
        # a thousand prompts come in at once, some behind rows that are there already
        dict(name="pages-prompts", op="pages", batch=1024, seq_lo=33, seq_hi=4608, new_lo=32, new_hi=512, pad=77,
             shape_seed=25),
        # the step's K and V rows of 128 requests
        dict(name="rows-step", op="rows", batch=128, hkv=8, d=128, dtype="bf16", seq_lo=33, seq_hi=2000, new_lo=1,
             new_hi=1, pad=0, shape_seed=26),
        # prompts of 64 requests stored at once, out of a fused qkv projection
        dict(name="rows-prompts", op="rows", batch=64, hkv=32, d=128, dtype="bf16", seq_lo=256, seq_hi=600, new_lo=100,
             new_hi=256, pad=9, shape_seed=27),
        # eight answers behind one instruction: few units, latency counts
        dict(name="shared-few", op="shared", mode="dense", batch=8, groups=1, hq=32, hkv=8, d=128, prefix_lo=1500,
             prefix_hi=1500, rest_lo=1, rest_hi=300, shape_seed=28),
        # 64 answers behind one long document
        dict(name="shared-long", op="shared", mode="dense", batch=64, groups=1, hq=32, hkv=8, d=128, prefix_lo=16391,
             prefix_hi=16391, rest_lo=1, rest_hi=600, shape_seed=29),
        # mixed serving: 128 requests of nine prompts, some alone
        dict(name="shared-mixed", op="shared", mode="dense", batch=128, groups=9, hq=32, hkv=8, d=128, prefix_lo=32,
             prefix_hi=2000, rest_lo=1, rest_hi=1024, shape_seed=30),
        # sixteen 32x32 images for each of four prompts, a mask for each head
        dict(name="shared-images", op="shared", mode="masked", batch=64, groups=4, hq=32, hkv=32, d=128, prefix_lo=256,
             prefix_hi=256, rest_lo=64, rest_hi=1024, window=96, keep=0.375, shape_seed=31),
        # 24x24 images of two prompts that end inside a page
        dict(name="shared-images-64", op="shared", mode="masked", batch=32, groups=2, hq=20, hkv=20, d=64, prefix_lo=120,
             prefix_hi=120, rest_lo=1, rest_hi=576, window=48, keep=0.2, shape_seed=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pages", "pages", "rows", "rows", "shared", "shared", "shared", "shared"])
    c = dict(op=op, shape_seed=rng.randrange(1 << 30))
    if op == "pages":
        c["batch"] = _log(rng, 1, 1024)
        n = _log(rng, 1, min(4000, 270_000 // c["batch"]))
        c.update(new_lo=rng.choice([0, 1, n // 2, n]), new_hi=n, seq_lo=n, seq_hi=_log(rng, n, max(n + 1, 4608)),
                 pad=rng.choice([0, 1, _log(rng, 1, 500)]))
        return c
    g = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 5, 8, 20, 32])
    if hkv * g > 64:
        g = 1
    c.update(hkv=hkv, d=rng.choice([64, 128]))
    row = hkv * c["d"]
    if op == "norm":
        # at most the elements of the largest listed call
        c.update(hq=hkv * g, dtype=rng.choice(["bf16", "bf16", "f32"]), kind=rng.choice(["rms", "rms", "layer"]),
                 per_head=rng.choice([False, True]), axes=rng.choice([1, 2, 3, 4]),
                 pairing=rng.choice(["halves", "neighbours"]), far=_log(rng, 64, 1 << 24),
                 tokens=_log(rng, 1, min(65096, 150_000_000 // (row * (g + 1)))))
        return c
    if op == "rows":
        c["batch"] = _log(rng, 1, 128)
        n = _log(rng, 1, max(1, min(4096, 45_000_000 // (row * c["batch"]))))
        c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), new_lo=rng.choice([0, n // 2, n]), new_hi=n, seq_lo=n,
                 seq_hi=_log(rng, n, n + 600), pad=rng.choice([0, 1, 50]))
        return c
    c.update(hq=hkv * g, mode=rng.choice(["dense", "masked"]), batch=_log(rng, 1, 128))
    c["groups"] = min(c["batch"], _log(rng, 1, 24))
    top = max(32, min(16391, 500_000_000 // (row * c["batch"])))
    p = _log(rng, 1, top)
    c.update(prefix_lo=rng.choice([0, p // 2, p]), prefix_hi=p)
    r = _log(rng, 1, max(16, min(4096, 250_000_000 // (row * c["batch"]))))
    c.update(rest_lo=rng.choice([0, 1, r // 2, r]), rest_hi=r)
    if c["prefix_lo"] + c["rest_lo"] < 1:
        c["rest_lo"] = 1
    if c["mode"] == "masked":
        c.update(window=rng.choice([0, 1, _log(rng, 2, 400), _log(rng, 2, 1000)]), keep=rng.choice([0.1, 0.375, 0.7]))
    return c


# ---------------------------------------------------------------------------
# sizes of a case
# ---------------------------------------------------------------------------

def _lengths(case):
    """Per-request lengths (and groups and masks) of a case, on the host."""
    rng = np.random.default_rng(case["shape_seed"])
    B = case["batch"]
    if case["op"] != "shared":
        L = rng.integers(case["seq_lo"], case["seq_hi"] + 1, size=B)
        return dict(L=L, n=np.minimum(rng.integers(case["new_lo"], case["new_hi"] + 1, size=B), L))
    G = case["groups"]
    cuts = np.sort(rng.choice(np.arange(1, B), size=G - 1, replace=False)) if G > 1 else np.zeros(0, int)
    start = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    of = np.repeat(np.arange(G), np.diff(start))
    S = rng.integers(case["prefix_lo"], case["prefix_hi"] + 1, size=G)[of]
    L = S + rng.integers(case["rest_lo"], case["rest_hi"] + 1, size=B)
    L = np.maximum(L, 1)
    out = dict(L=L, S=S, start=start, of=of)
    if case["mode"] == "masked":
        # the prompt ends with the prefix, or goes on behind it
        W = case["window"]
        out["P"] = S + np.where(rng.random(B) < 0.25, rng.integers(0, 40, size=B), 0)
        out["W"] = rng.integers(W // 2, W + 1, size=B)
        keep = rng.random((B, case["hkv"], max(W, 1))) < case["keep"]
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


def _kept_rest(s):
    """Rows behind the prefix that the query of each request keeps, [B, hkv]."""
    L, P, W, S = s["L"], s["P"], s["W"], s["S"]
    npr = np.minimum(P, L)
    reach = np.where(L - 1 >= npr, np.minimum(L - 1 - npr, W), -1)
    cum = np.concatenate([np.zeros(s["keep"].shape[:2] + (1,), np.int64), np.cumsum(s["keep"], axis=2)], axis=2)
    win = np.take_along_axis(cum, np.clip(reach, 0, cum.shape[2] - 1)[:, None, None], axis=2)[:, :, 0]
    return (npr - S)[:, None] + np.where(reach[:, None] >= 0, win + 1, 0)


def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * e + 4 * case["tokens"] * case["axes"], "flops": 8 * n}
    s = _lengths(case)
    if op == "pages":
        n = int(s["n"].sum())
        pages = int(((s["L"] + PAGE - 1) // PAGE - (s["L"] - s["n"] + PAGE - 1) // PAGE).sum())
        return {"bytes": 12 * case["batch"] + 8 * (n + case["pad"]) + 8 * pages, "flops": 0}
    row = case["hkv"] * case["d"]
    if op == "rows":
        n, e = int(s["n"].sum()), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4 * n * row * e + 4 * (n + case["pad"]), "flops": 0}
    rest = int((s["L"] - s["S"]).sum()) * case["hkv"] if case["mode"] == "dense" else int(_kept_rest(s).sum())
    prefix = s["S"][s["start"][:-1]]
    pairs = int(s["S"].sum()) * case["hkv"] + rest
    qo = case["batch"] * case["hq"] * (2 * case["d"] * 2 + 4)
    return {"bytes": 4 * (int(prefix.sum()) * row + rest * case["d"]) + qo,
            "flops": 4 * pairs * (case["hq"] // case["hkv"]) * case["d"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


def _positions(case):
    """[tokens, axes] positions: runs of text (every axis alike), then image tokens (the last two axes run)."""
    rng = np.random.default_rng(case["shape_seed"])
    n, axes = case["tokens"], case["axes"]
    base = np.repeat(rng.integers(0, case["far"], size=1 + n // 8192), 8192)[:n]
    k = np.arange(n) % 8192
    run_of = {axes - 2: k // 90, axes - 1: k % 90 if axes > 1 else k}
    pos = np.stack([base + run_of.get(a, 0) for a in range(axes)], axis=1)
    pos[k < 64] = (base + k)[k < 64][:, None]
    return pos


def _pair_axis(case):
    """Axis of each pair, whole blocks: the first axis turns what the others leave."""
    half, axes = case["d"] // 2, case["axes"]
    each = half // (axes + 1) if axes > 1 else 0
    return [0] * (half - each * (axes - 1)) + [a for a in range(1, axes) for _ in range(each)]


def _inv_freq(d):
    return [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]


EPS = 1e-6


def _table(pages_of, ids, width):
    """A page table: pages_of[b] are the indices of request b's pages in ids."""
    table = np.full((len(pages_of), width), -1, dtype=np.int64)
    for b, p in enumerate(pages_of):
        table[b, :len(p)] = p
    idx = torch.as_tensor(table, device="cuda")
    return torch.where(idx >= 0, ids[idx.clamp(min=0)], torch.full_like(idx, -1).to(torch.int32)).contiguous()


def _own_pages(counts):
    at = np.concatenate([[0], np.cumsum(counts)])
    return [np.arange(at[b], at[b + 1]) for b in range(len(counts))], int(at[-1])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda shape, dt: torch.randn(shape, generator=gen, device="cuda").to(dt)  # noqa: E731
    op = case["op"]
    if op == "norm":
        n, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
        # heads differ in size, as a projection's do
        size = torch.exp(0.7 * torch.randn((1, hq + 2 * hkv, 1), generator=gen, device="cuda"))
        qkv = (torch.randn((n, hq + 2 * hkv, d), generator=gen, device="cuda") * size).to(dt)
        st = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], positions=_i32(_positions(case)),
                  q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"),
                  k_out=torch.empty((n, hkv, d), dtype=dt, device="cuda"))
        for x, heads in (("q", hq), ("k", hkv)):
            shape = (heads, d) if case["per_head"] else (d,)
            st[x + "_weight"] = (1 + 0.2 * randn(shape, torch.float32)).to(dt)
            st[x + "_bias"] = (0.1 * randn(shape, torch.float32)).to(dt) if case["kind"] == "layer" else None
        return st
    s = _lengths(case)
    if op in ("pages", "rows"):
        L, n = s["L"], s["n"]
        have, all_ = (L - n + PAGE - 1) // PAGE, (L + PAGE - 1) // PAGE
        width, total = int(all_.max()) + 3, int(n.sum())
    if op == "pages":
        mapped, used = _own_pages(have)
        need = int((all_ - have).sum())
        pool = used + need + 40
        ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        most = total + case["pad"]
        free = torch.cat([ids[used:], torch.full((9,), -7, dtype=torch.int32, device="cuda")])
        return dict(case=case, seq_len=_i32(L), new_len=_i32(n), page_table=_table(mapped, ids, width), free=free,
                    count=_i32([pool - used]), pool=pool,
                    count_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    token_start=torch.zeros(len(L) + 1, dtype=torch.int32, device="cuda"),
                    row_slot=torch.zeros(most, dtype=torch.int32, device="cuda"),
                    row_pos=torch.zeros(most, dtype=torch.int32, device="cuda"))
    hkv, d = case["hkv"], case["d"]
    if op == "rows":
        dt = DTYPES[case["dtype"]]
        mapped, pool = _own_pages(all_)
        ids = torch.randperm(pool + 2, generator=gen, device="cuda").to(torch.int32)
        at = np.concatenate([np.arange(L[b] - n[b], L[b]) for b in range(len(L))] + [np.zeros(case["pad"], int)])
        of = np.repeat(np.arange(len(L)), n)
        page = np.concatenate([mapped[b][(np.arange(L[b] - n[b], L[b])) // PAGE] for b in range(len(L))]).astype(np.int64)
        slot = ids.long()[torch.as_tensor(page, device="cuda")] * PAGE + torch.as_tensor(at[:len(of)] % PAGE, device="cuda")
        slot = torch.cat([slot, torch.full((case["pad"],), -1, dtype=slot.dtype, device="cuda")]).to(torch.int32)
        qkv = randn((len(slot), 3 * hkv, d), dt)
        return dict(case=case, row_slot=slot, k=qkv[:, hkv:2 * hkv], v=qkv[:, 2 * hkv:],
                    k_pages=randn((pool + 2, PAGE, hkv, d), dt), v_pages=randn((pool + 2, PAGE, hkv, d), dt))
    # shared: the whole pages of a group's prefix are the same pages; a page that ends inside the
    # prefix is copied for every request, as its own rows follow in it
    L, S, B = s["L"], s["S"], case["batch"]
    pages_of, at, copies = [], 0, []
    for g in range(case["groups"]):
        b0, b1 = int(s["start"][g]), int(s["start"][g + 1])
        whole, part = int(S[b0]) // PAGE, int(S[b0]) % PAGE
        shared = np.arange(at, at + whole)
        at += whole
        for b in range(b0, b1):
            n = (int(L[b]) + PAGE - 1) // PAGE - whole
            pages_of.append(np.concatenate([shared, np.arange(at, at + n)]))
            if part and b > b0:
                copies.append((int(pages_of[b0][whole]), at, part))
            at += n
    ids = torch.randperm(at + 3, generator=gen, device="cuda").to(torch.int32)
    st = dict(case=case, page_table=_table(pages_of, ids, max(len(p) for p in pages_of)), seq_len=_i32(L),
              prefix_len=_i32(S), group_start=_i32(s["start"]), longest=int(L.max()), pool=at + 3,
              max_prefix=int(S.max()), max_rest=int((L - S).max()) if case["mode"] == "dense" else int(_kept_rest(s).max()),
              scale=1.0 / math.sqrt(d))
    for x in ("k", "v"):
        t = torch.randn((at + 3, PAGE, hkv, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        if copies:
            src, dst, part = (torch.as_tensor(c, device="cuda") for c in zip(*copies))
            rows = torch.arange(PAGE, device="cuda") < part[:, None]
            src, dst = ids.long()[src], ids.long()[dst]
            t[dst] = torch.where(rows[:, :, None, None], t[src], t[dst])
        st[x] = t
    if case["mode"] == "masked":
        W = case["window"]
        st.update(prompt_len=_i32(s["P"]), window=_i32(s["W"]),
                  keep_mask=torch.as_tensor(_bits(s["keep"], _words(W)).view(np.int32), device="cuda"))
    st["q"] = randn((B, case["hq"], d), torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((B, case["hq"]), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _norm_plain(st):
    case, d = st["case"], st["case"]["d"]
    axis = torch.tensor(_pair_axis(case), device="cuda")
    freq = torch.tensor(_inv_freq(d), dtype=torch.float64, device="cuda")
    angle = st["positions"][:, axis].double() * freq            # far positions: the angle in 64 bits
    turn = 2 * math.pi
    angle = (angle - turn * torch.floor(angle / turn)).float()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    outs = {}
    for name in ("q", "k"):
        x = st[name].float()
        if case["kind"] == "layer":
            x = x - x.mean(-1, keepdim=True)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * st[name + "_weight"].float()
        if st[name + "_bias"] is not None:
            x = x + st[name + "_bias"].float()
        if case["pairing"] == "halves":
            a, b = x[..., :d // 2], x[..., d // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        outs[name] = y.to(DTYPES[case["dtype"]])
    return outs


def _pages_plain(st):
    L, n = st["seq_len"].long(), st["new_len"].long()
    B, most = L.shape[0], st["row_slot"].shape[0]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    start = torch.cat([zero, n.cumsum(0)])
    first = (L - n + PAGE - 1) // PAGE                          # the first page whose rows are all new
    need = (L + PAGE - 1) // PAGE - first
    before = need.cumsum(0) - need
    t = torch.arange(most, device="cuda")
    live = t < start[-1]
    steps = torch.zeros(most + 1, dtype=torch.int64, device="cuda")
    steps = steps.index_add(0, start[1:B].clamp(max=most), torch.ones(B - 1, dtype=torch.int64, device="cuda"))
    b = steps[:most].cumsum(0)
    row = torch.where(live, (L - n)[b] + t - start[b], torch.zeros_like(t))
    page = row // PAGE
    fresh = live & (page >= first[b])
    take = st["count"].long() - 1 - (before[b] + page - first[b])
    had = st["page_table"].long()[b, page]
    got = torch.where(fresh, st["free"].long()[torch.where(fresh, take, torch.zeros_like(take))], had)
    # every row of a page writes the page's id, the rows behind the last one to a place past the table
    width, size = st["page_table"].shape[1], st["page_table"].numel()
    table = torch.cat([st["page_table"].view(-1), torch.zeros(1, dtype=torch.int32, device="cuda")])
    table[torch.where(live, b * width + page, torch.full_like(b, size))] = got.to(torch.int32)
    table = table[:size].view(-1, width)
    return {"page_table": table, "free_count": (st["count"] - need.sum()).to(torch.int32),
            "token_start": start.to(torch.int32),
            "row_slot": torch.where(live, got * PAGE + row % PAGE, torch.full_like(row, -1)).to(torch.int32),
            "row_pos": row.to(torch.int32)}


def _rows_plain(st):
    on = st["row_slot"] >= 0
    at = st["row_slot"].long()[on]
    for x in ("k", "v"):
        st[x + "_pages"].flatten(0, 1)[at] = st[x][on]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _kept(st):
    """Whether the query of each request keeps row j: [B, hkv, longest]."""
    j = torch.arange(st["longest"], device="cuda")
    L, P, W = st["seq_len"].long()[:, None], st["prompt_len"].long()[:, None], st["window"].long()[:, None]
    o = L - 1 - j
    B, hkv, words = st["keep_mask"].shape
    bit = (o - 1).clamp(min=0)
    at = (bit // 32).clamp(max=words - 1)[:, None].expand(B, hkv, -1)
    on = ((torch.gather(st["keep_mask"].long(), 2, at) >> (bit % 32)[:, None]) & 1) != 0
    return ((o >= 0) & ((j < P) | (o == 0)))[:, None] | (((o >= 1) & (o <= W) & (j >= P))[:, None] & on)


def _shared_plain(st):
    case, B = st["case"], st["case"]["batch"]
    hkv, d = case["hkv"], case["d"]
    b = torch.arange(B, device="cuda")[:, None]
    j = torch.arange(st["longest"], device="cuda").expand(B, -1)
    live = j < st["seq_len"].long()[:, None]
    j = torch.where(live, j, torch.zeros_like(j))
    keep = live[:, None] if case["mode"] == "dense" else _kept(st)
    page = st["page_table"].long()[b, j // PAGE]
    s = torch.matmul(st["q"].float().view(B, hkv, -1, d), st["k"][page, j % PAGE].float().permute(0, 2, 3, 1))
    s = torch.where(keep[:, :, None], s * st["scale"], torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, st["v"][page, j % PAGE].float().transpose(1, 2)) / total
    return {"out": out.reshape(B, -1, d).to(torch.bfloat16), "lse": (m + torch.log(total)).reshape(B, -1)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _handle(st):
    """What a program keeps beside its cache: the dims, the workspace, the norm and the groups."""
    if "handle" not in st:
        from kv_cache_serving_gb300 import dsa
        c = st["case"]
        op = c["op"]
        if op == "norm":
            dims = dsa.make_dims(1, c["hq"], c["hkv"], c["d"], 1, 1, 0, 1, 1, c["dtype"], c["dtype"])
            rope = dsa.make_rope(_inv_freq(c["d"]), _pair_axis(c), pairing=c["pairing"], axes=c["axes"])
            norm = dsa.make_qk_norm(c["kind"], EPS, st["q_weight"], st["k_weight"], st["q_bias"], st["k_bias"])
            st["handle"] = (dsa, dims, norm, rope)
        elif op == "pages":
            dims = dsa.make_dims(c["batch"], 1, 1, 64, st["pool"], st["page_table"].shape[1], 0, 1, 1, "bf16", "bf16")
            st["handle"] = (dsa, dims, dsa.alloc_workspace(dims))
        elif op == "rows":
            dims = dsa.make_dims(c["batch"], c["hkv"], c["hkv"], c["d"], st["k_pages"].shape[0], 1, 0, 1, 1, c["dtype"],
                                 c["dtype"])
            st["handle"] = (dsa, dims, dsa.alloc_workspace(dims))
        else:
            W = c.get("window", 0)
            dims = dsa.make_dims(c["batch"], c["hq"], c["hkv"], c["d"], st["pool"], st["page_table"].shape[1], W,
                                 _words(W), st["max_prefix"] + st["max_rest"], "bf16", "bf16")
            shared = dsa.shared_prefix(st["group_start"], st["prefix_len"], st["max_prefix"], st["max_rest"])
            st["handle"] = (dsa, dims, shared, dsa.alloc_workspace(dims))
    return st["handle"]


def _run_own(st):
    op = st["case"]["op"]
    if op == "norm":
        dsa, dims, norm, rope = _handle(st)
        dsa.dsa_qk_norm_rope(dims, norm, rope, st["positions"], st["q"], st["k"], st["q_out"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "pages":
        dsa, dims, ws = _handle(st)
        dsa.dsa_assign_pages(dims, st["seq_len"], st["new_len"], st["free"], st["count"], st["count_out"],
                             st["page_table"], st["token_start"], st["row_slot"], st["row_pos"], ws)
        return {"page_table": st["page_table"], "free_count": st["count_out"], "token_start": st["token_start"],
                "row_slot": st["row_slot"], "row_pos": st["row_pos"]}
    if op == "rows":
        dsa, dims, ws = _handle(st)
        dsa.dsa_write_rows(dims, st["row_slot"], st["k"], st["v"], st["k_pages"], st["v_pages"], ws)
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    dsa, dims, shared, ws = _handle(st)
    if st["case"]["mode"] == "dense":
        dsa.dsa_decode_dense_shared(dims, shared, st["q"], st["k"], st["v"], st["page_table"], st["seq_len"],
                                    st["scale"], st["out"], st["lse"], ws)
    else:
        dsa.dsa_decode_sparse_masked_shared(dims, shared, st["q"], st["k"], st["v"], st["page_table"], st["seq_len"],
                                            st["prompt_len"], st["window"], st["keep_mask"], st["scale"], st["out"],
                                            st["lse"], ws)
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "pages": _pages_plain, "rows": _rows_plain, "shared": _shared_plain}[
        state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(st):
    case, d = st["case"], st["case"]["d"]
    pos = st["positions"].double()
    angle = torch.stack([pos[:, a] * 10000.0 ** (-2.0 * i / d) for i, a in enumerate(_pair_axis(case))], dim=1)
    half = case["pairing"] == "halves"
    lo, hi = (slice(0, d // 2), slice(d // 2, d)) if half else (slice(0, d, 2), slice(1, d, 2))
    out = {}
    for name in ("q", "k"):
        x, w, c = st[name].double(), st[name + "_weight"].double(), st[name + "_bias"]
        mean = x.sum(-1, keepdim=True) / d if case["kind"] == "layer" else 0.0
        size = ((x - mean) ** 2).sum(-1, keepdim=True) / d + EPS
        x = (x - mean) * size ** -0.5 * w + (0.0 if c is None else c.double())
        z = torch.polar(torch.ones_like(angle), angle)[:, None] * torch.complex(x[..., lo], x[..., hi])
        y = torch.empty_like(x)
        y[..., lo], y[..., hi] = z.real, z.imag
        out[name] = y
    return out


def _exact_rows(st):
    """Nothing is rounded: the rows as they are."""
    n = st["row_slot"].shape[0] - st["case"]["pad"]             # the rows behind have no slot
    out = {}
    for x in ("k", "v"):
        pages = st[x + "_pages"].double()
        pages.flatten(0, 1).index_copy_(0, st["row_slot"][:n].long(), st[x][:n].double())
        out[x + "_pages"] = pages
    return out


def _exact_shared(st):
    """Request by request: softmax over its kept rows, read through its own page table."""
    case = st["case"]
    hkv, d, g = case["hkv"], case["d"], case["hq"] // case["hkv"]
    L, table = st["seq_len"].tolist(), st["page_table"].long()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        n = L[b]
        pages = table[b, :(n + PAGE - 1) // PAGE]
        k, v = (st[x][pages].flatten(0, 1)[:n].double() for x in ("k", "v"))         # [n, hkv, d]
        on = torch.ones((hkv, n), dtype=torch.bool, device="cuda")
        if case["mode"] == "masked":
            p, w = int(st["prompt_len"][b]), int(st["window"][b])
            off = n - 1 - np.arange(n)
            words = st["keep_mask"][b].cpu().numpy().view(np.uint32)
            bit = np.maximum(off - 1, 0)
            set_ = (words[:, np.minimum(bit // 32, words.shape[1] - 1)] >> (bit % 32).astype(np.uint32)) & 1
            keep = (np.arange(n) < p) | (off == 0) | ((off >= 1) & (off <= w) & (set_ != 0))
            on = torch.as_tensor(keep, device="cuda")
        q = st["q"][b].double().view(hkv, g, d)
        x = torch.einsum("hgd,nhd->hgn", q, k) * st["scale"]
        x = x.masked_fill(~on[:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        out[b] = torch.einsum("hgn,nhd->hgd", torch.exp(x - z[..., None]), v).reshape(-1, d)
        lse[b] = z.reshape(-1)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers
    st = prepare(case, seed)
    return {"norm": _exact_norm, "rows": _exact_rows, "shared": _exact_shared}[case["op"]](st)
