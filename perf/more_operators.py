"""The operators of drafting and of page keeping over the paged KV cache, as cases to be measured.

A server that drafts verifies a tree of tokens for every request at once, keeps those that the
model agrees with and gives the others' rows and pages back; requests fork and end in between:

  plan     tree_plan: positions and ancestor masks of the drafted tokens, from their parents
  attn     tree_attn: attention of the drafted tokens over a shared prefix, their requests' cached
           keys and their own ancestors in the tree
  compact  cache_compact: kept rows move together in the pages, in all layers; new lengths
  free     page_free: requests that end or are cut back give their pages back
  beam     page_free of the beams that lost, then page_fork of those that won into their rows: full
           pages are shared, the partial one is copied in all layers

`own` False: plain torch, 32 bits, rounded once at the end.  `own` True: the package's calls.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"


def _dt(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def listed():
    return [
        # ---- plan -----------------------------------------------------------------------------
        # eight requests with a tree of 16 tokens each: latency alone
        {"name": "plan_8x16", "op": "plan", "R": 8, "lo": 16, "hi": 16, "tree": 16, "width": 3, "cached": 32768, "pad": 0},
        # a busy server: 1000 requests, trees of 1 to 64 tokens, batch padded
        {"name": "plan_1000x64", "op": "plan", "R": 1000, "lo": 1, "hi": 64, "tree": 64, "width": 4, "cached": 8000, "pad": 500},
        # ---- attn -----------------------------------------------------------------------------
        # one request of 1000 tokens with a tree of 8: latency alone
        {"name": "attn_one_1000", "op": "attn", "dtype": BF16, "R": 1, "lo": 8, "hi": 8, "width": 3, "Hq": 64, "Hkv": 8, "d": 128, "page": 64,
         "prefix": 0, "own_lo": 1000, "own_hi": 1000},
        # 48 requests behind a 32768-token document, trees of 5 to 25 tokens, up to 2000 cached tokens of their own
        {"name": "attn_prefix_32768", "op": "attn", "dtype": BF16, "R": 48, "lo": 5, "hi": 25, "width": 4, "Hq": 64, "Hkv": 8, "d": 128, "page": 64,
         "prefix": 32768, "own_lo": 4, "own_hi": 2000},
        # 16 long requests with trees of 64: many rows for each key
        {"name": "attn_64_32768", "op": "attn", "dtype": BF16, "R": 16, "lo": 64, "hi": 64, "width": 6, "Hq": 64, "Hkv": 8, "d": 128, "page": 128,
         "prefix": 0, "own_lo": 8192, "own_hi": 32768},
        # 32 bits, small heads, an odd prefix
        {"name": "attn_f32_4097", "op": "attn", "dtype": F32, "R": 5, "lo": 3, "hi": 13, "width": 2, "Hq": 8, "Hkv": 4, "d": 64, "page": 32,
         "prefix": 4097, "own_lo": 2, "own_hi": 500},
        # ---- compact --------------------------------------------------------------------------
        # after a step of 64 requests: up to 6 of 48 drafted tokens are kept, in 16 layers
        {"name": "compact_tree_64", "op": "compact", "dtype": BF16, "R": 64, "layers": 16, "Hkv": 8, "d": 128, "page": 64, "own_lo": 100,
         "own_hi": 600, "tree": 48, "keep": 6, "window": False},
        # a sliding window: four caches of up to 24576 tokens keep their first 4 and newest 8188 tokens, in 4 layers
        {"name": "compact_window_8192", "op": "compact", "dtype": BF16, "R": 4, "layers": 4, "Hkv": 8, "d": 128, "page": 64, "own_lo": 16384,
         "own_hi": 24576, "tree": 0, "keep": 8192, "window": True},
        # ---- free -----------------------------------------------------------------------------
        # eight requests take back the pages of their rejected tokens
        {"name": "free_cut_8", "op": "free", "R": 8, "page": 64, "lo": 100, "hi": 32768, "ends": 0.0, "cut": 64},
        # 4000 requests, a third of them has ended, the others are cut back a little
        {"name": "free_ends_4000", "op": "free", "R": 4000, "page": 16, "lo": 10, "hi": 4000, "ends": 0.33, "cut": 20},
        # ---- beam -----------------------------------------------------------------------------
        # four of eight beams go on, each into the row of one that lost, in 8 layers
        {"name": "beam_8", "op": "beam", "dtype": BF16, "R": 8, "forks": 4, "layers": 8, "Hkv": 8, "d": 128, "page": 64, "lo": 1000, "hi": 4000},
        # 16 prompts, 15 samples of each started anew, small pages, an odd number of key heads, 24 layers
        {"name": "beam_256", "op": "beam", "dtype": BF16, "R": 256, "forks": 240, "layers": 24, "Hkv": 5, "d": 128, "page": 128, "lo": 300, "hi": 2000},
    ]


# What a drawn case may cost at most: the largest listed one's bytes and operations.
_MOST = {}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["plan", "attn", "attn", "compact", "free", "beam"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = _log(rng, 1, 256)
        return {"op": op, "R": _log(rng, 1, 1000), "lo": rng.choice([1, hi]), "hi": hi, "tree": hi + rng.choice([0, 0, 5]), "width": rng.choice([1, 2, 4, 8]),
                "cached": _log(rng, 1, 40000), "pad": rng.randrange(0, 500)}
    if op == "free":
        return {"op": op, "R": _log(rng, 1, 4000), "page": page, "lo": _log(rng, 1, 1000), "hi": _log(rng, 1000, 40000),
                "ends": rng.choice([0.0, 0.1, 0.5, 1.0]), "cut": _log(rng, 1, 300)}
    dtype = rng.choice([BF16, BF16, F32])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 8])
    if op == "compact":
        window = rng.random() < 0.4
        keep = _log(rng, 16, 8192) if window else _log(rng, 1, 16)
        lo = 2 * keep + rng.randrange(0, 100) if window else _log(rng, 1, 500)
        return {"op": op, "dtype": dtype, "R": _log(rng, 1, 100), "layers": _log(rng, 1, 24), "Hkv": Hkv, "d": d, "page": page, "own_lo": lo,
                "own_hi": int(lo * rng.uniform(1, 2)), "tree": 0 if window else 2 * keep + rng.randrange(0, 60), "keep": keep, "window": window}
    if op == "beam":
        R = _log(rng, 2, 256)
        lo = _log(rng, 10, 1000)
        return {"op": op, "dtype": dtype, "R": R, "forks": rng.randint(1, R - 1), "layers": _log(rng, 1, 24), "Hkv": Hkv, "d": d, "page": page,
                "lo": lo, "hi": int(lo * rng.uniform(1, 4))}
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    small = dtype == F32  # the 32-bit path is for short contexts
    hi = _log(rng, 1, 24 if small else 200)
    own_hi = _log(rng, 1, 1000 if small else 32768)
    return {"op": op, "dtype": dtype, "R": _log(rng, 1, 8 if small else 64), "lo": rng.choice([1, hi]), "hi": hi, "width": rng.choice([1, 2, 4, 8]),
            "Hq": G * Hkv, "Hkv": Hkv, "d": d, "page": page, "prefix": rng.choice([0, 1]) * _log(rng, 1, 8000 if small else 32768),
            "own_lo": max(1, own_hi // 8), "own_hi": own_hi}


def _size(case):
    """Values that the plain form holds at once."""
    op = case["op"]
    if op == "attn":
        return case["R"] * case["hi"] * case["Hq"] * (case["prefix"] + case["own_hi"] + case["hi"])
    if op == "plan":
        return case["R"] * case["hi"] ** 2
    if op == "free":
        return case["R"] * case["hi"] // case["page"]
    if op == "compact":
        pages = sum(_pages(n, case["page"]) for n in _compact_lens(case)[1])
    else:
        lens, src, _ = _beam_plan(case)
        pages = sum(_pages(n, case["page"]) for n in lens[: case["R"] - case["forks"]]) + len(src)
    return pages * case["page"] * case["layers"] * case["Hkv"] * case["d"] * (2 if case["dtype"] == F32 else 1)


def draw(rng):
    if not _MOST:
        for c in listed():
            w = work(c)
            m = _MOST.setdefault((c["op"], c.get("dtype", "") if c["op"] == "attn" else ""), {"bytes": 0, "flops": 0, "size": 0})
            for k, x in (("bytes", w["bytes"]), ("flops", w["flops"]), ("size", _size(c))):
                m[k] = max(m[k], x)
    while True:
        c = _drawn(rng)
        m, w = _MOST[(c["op"], c.get("dtype", "") if c["op"] == "attn" else "")], work(c)
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _size(c) <= m["size"]:
            return c


# ---- lengths: plain numbers that follow from the case alone -----------------------------------------


def _rng(case):
    return random.Random(" ".join("%s=%s" % kv for kv in sorted(case.items()) if kv[0] != "name"))


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) if hi > lo else lo


def _tree_sizes(case):
    r = _rng(case)
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["R"])]
    n[-1] = case["hi"]
    return n


def _attn_lens(case):
    """Cached tokens of every request, without its drafted ones."""
    r = _rng(dict(case, of="lens"))
    lens = [_spread(r, case["own_lo"], case["own_hi"]) for _ in range(case["R"])]
    lens[0] = case["own_hi"]
    return lens


def _compact_lens(case):
    """(tokens that stay where they are, all tokens, tokens kept of the others) of every request."""
    r = _rng(case)
    if case["window"]:
        lens = [r.randint(case["own_lo"], case["own_hi"]) for _ in range(case["R"])]
        return [0] * case["R"], lens, [case["keep"]] * case["R"]
    base = [_spread(r, case["own_lo"], case["own_hi"]) for _ in range(case["R"])]
    kept = [r.randint(0, case["keep"]) for _ in base]
    kept[-1] = case["keep"]
    return base, [b + case["tree"] for b in base], kept


def _free_lens(case):
    r = _rng(case)
    lens = [_spread(r, case["lo"], case["hi"]) for _ in range(case["R"])]
    keep = [0 if r.random() < case["ends"] else max(0, n - r.randint(0, case["cut"])) for n in lens]
    keep[0] = max(0, lens[0] - case["cut"])
    return lens, keep


def _beam_plan(case):
    """(lengths, forks' sources and destinations): rows [0, R - forks) go on, the others take their tokens."""
    r = _rng(case)
    R, F = case["R"], case["forks"]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(R)]
    src = [r.randrange(R - F) for _ in range(F)]
    dst = list(range(R - F, R))
    r.shuffle(dst)
    for a, b in zip(src, dst):
        lens[b] = lens[a]
    return lens, src, dst


def _pages(n, page):
    return -(-n // page)


# ---- inputs -----------------------------------------------------------------------------------------


class _State(dict):
    __getattr__ = dict.__getitem__
    __setattr__ = dict.__setitem__


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _State(case)
    return {"plan": _prepare_plan, "attn": _prepare_attn, "compact": _prepare_compact, "free": _prepare_free, "beam": _prepare_beam}[case["op"]](case, s, g)


def _cu(counts):
    return _i32([0] + torch.cumsum(torch.tensor(counts), 0).tolist())


def _tables(counts, ids, width):
    """Block tables whose rows take their pages from `ids` one after the other; -1 behind them."""
    at = _cu(counts).long()
    col = torch.arange(width, device="cuda")
    return torch.where(col < torch.tensor(counts, device="cuda")[:, None], ids[(at[:-1, None] + col).clamp_(max=ids.numel() - 1)],
                       torch.full((), -1, dtype=torch.int32, device="cuda")).to(torch.int32).contiguous()


def _parents(sizes, width, g):
    """A drafted forest's parents, in the order of drafting: one of the `width` tokens before, -1 for none."""
    i = torch.cat([torch.arange(n) for n in sizes]).cuda()
    u = torch.rand(i.numel(), generator=g, device="cuda")
    return (i - 1 - (u * width).long().clamp_(max=width - 1)).clamp_(min=-1).int()


def _closure(parent, cu, n):
    """Ancestors-or-self [R, n, n] of forests padded to n tokens."""
    R = cu.numel() - 1
    r = torch.searchsorted(cu[1:], torch.arange(parent.numel(), device="cuda"), right=True)
    live = r < R
    r, p = r[live], parent[live].long()
    i = torch.arange(parent.numel(), device="cuda")[live] - cu[r]
    m = torch.zeros(R, n, n + 1, device="cuda")  # (the last column takes the parent of the roots)
    m[r, i, torch.where(p < 0, n, p)] = 1
    m = m[:, :, :n] + torch.eye(n, device="cuda")
    for _ in range(max(1, (n - 1).bit_length())):  # 2^k generations after k products
        m = (m @ m).clamp_(max=1)
    return m


def _packed(m, r, i, words):
    """Bits of rows (r, i) of `m` as 32-bit words."""
    bits = torch.nn.functional.pad(m[r, i], (0, words * 32 - m.shape[2])).view(-1, words, 32).long()
    w = (bits << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def _prepare_plan(case, s, g):
    sizes = _tree_sizes(case)
    s.cu = _cu(sizes)
    pad = torch.full((case["pad"],), 7, dtype=torch.int32, device="cuda")  # what a padded batch holds there
    s.parent = torch.cat([_parents(sizes, case["width"], g), pad])
    s.kv_len = torch.randint(0, case["cached"] + 1, (case["R"],), generator=g, device="cuda", dtype=torch.int32) + _i32(sizes)
    return s


def _prepare_attn(case, s, g):
    R, Hq, Hkv, d, dt, page = case["R"], case["Hq"], case["Hkv"], case["d"], _dt(case), case["page"]
    sizes, cached = _tree_sizes(case), _attn_lens(case)
    T = sum(sizes)
    counts = [_pages(c + n, page) for c, n in zip(cached, sizes)]
    np_prefix = _pages(case["prefix"], page)
    n_pages = np_prefix + sum(counts) + 3
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda", dtype=dt)  # noqa: E731
    s.q = randn(T, Hq, d)
    s.cache_k, s.cache_v = randn(n_pages, Hkv, page, d), randn(n_pages, Hkv, page, d)
    ids = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    s.prefix_pages = ids[:np_prefix].contiguous()
    s.table = _tables(counts, ids[np_prefix:], max(counts) + 1)
    s.kv_len, s.cu = _i32([c + n for c, n in zip(cached, sizes)]), _cu(sizes)
    s.longest, s.most = max(c + n for c, n in zip(cached, sizes)), max(sizes)
    parent = _parents(sizes, case["width"], g)
    s.r = torch.repeat_interleave(torch.arange(R), torch.tensor(sizes)).cuda()
    s.i = torch.arange(T, device="cuda") - s.cu.long()[s.r]
    s.mask = _packed(_closure(parent, s.cu, s.most), s.r, s.i, _pages(s.most, 32))  # the step's, of all its layers
    return s


def _caches(case, s, g, n_pages):
    shape = (case["layers"], n_pages, case["Hkv"], case["page"], case["d"])
    s.cache_k = torch.randn(shape, generator=g, device="cuda", dtype=_dt(case))
    s.cache_v = torch.randn(shape, generator=g, device="cuda", dtype=_dt(case))


def _prepare_compact(case, s, g):
    base, lens, kept = _compact_lens(case)
    counts = [_pages(n, case["page"]) for n in lens]
    n_pages = sum(counts) + 2
    s.table = _tables(counts, torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32), max(counts) + 1)
    s.base, s.kv_len, s.keep_len = _i32(base), _i32(lens), _i32(kept)
    n = case["keep"]
    i = torch.arange(n, device="cuda")
    if case["window"]:
        s.lists = torch.where(i < 4, i, s.kv_len.long()[:, None] - n + i).int().contiguous()
    else:
        # an accepted path: the first child or none of its siblings, then tokens behind the first levels
        u = torch.rand(case["R"], case["tree"] - n, generator=g, device="cuda")
        deep = u.argsort(1)[:, :n].sort(1).values + n
        first = torch.rand(case["R"], 1, generator=g, device="cuda") < 0.5
        s.lists = torch.where(first & (i == 0), 0, deep).int().contiguous()
    _caches(case, s, g, n_pages)
    return s


def _prepare_free(case, s, g):
    lens, keep = _free_lens(case)
    counts = [_pages(n, case["page"]) for n in lens]
    s.n_pages = sum(counts) + 100
    ids = torch.randperm(s.n_pages, generator=g, device="cuda", dtype=torch.int32)
    s.table = _tables(counts, ids, max(counts) + 1)
    s.kv_len, s.keep_len = _i32(lens), _i32(keep)
    s.free = torch.cat([ids.flip(0)[:100], ids[:-100]]).contiguous()  # the pool: what is in use lies before `start`
    s.free = torch.roll(s.free, -100)
    s.free_start = torch.tensor([s.n_pages - 100], dtype=torch.int64, device="cuda")
    return s


def _prepare_beam(case, s, g):
    lens, src, dst = _beam_plan(case)
    page, R, F = case["page"], case["R"], case["forks"]
    full, counts = [n // page for n in lens], [_pages(n, page) for n in lens]
    own_counts = [counts[r] if r < R - F else 0 for r in range(R)]
    fresh = [f for f in range(F) if lens[src[f]] % page]
    n_pages = sum(own_counts) + len(fresh) + 20
    ids = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    used = sum(own_counts)
    table = _tables(own_counts, ids, max(counts) + 1).cpu()
    # the rows as the step before left them: full pages shared, the partial one of their own, in ascending order
    taken = ids[used:used + len(fresh)].sort().values.cpu()
    shares = torch.zeros(n_pages, dtype=torch.int32)
    for f in range(F):
        table[dst[f], : full[src[f]]] = table[src[f], : full[src[f]]]
        shares.index_add_(0, table[src[f], : full[src[f]]].long(), torch.ones(full[src[f]], dtype=torch.int32))
    for i, f in enumerate(fresh):
        table[dst[f], full[src[f]]] = taken[i]
    s.n_pages, s.table, s.shares = n_pages, table.cuda(), shares.cuda()
    s.kv_len, s.src, s.dst = _i32(lens), _i32(src), _i32(dst)
    s.keep_len = s.kv_len.clone()
    s.keep_len[s.dst.long()] = 0
    s.free = torch.cat([ids[:used], taken.cuda(), ids[used + len(fresh):]]).contiguous()
    s.free_start = torch.tensor([used + len(fresh)], dtype=torch.int64, device="cuda")
    _caches(case, s, g, n_pages)
    return s


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    return {"plan": _run_plan, "attn": _run_attn, "compact": _run_compact, "free": _run_free, "beam": _run_beam}[s["op"]](s)


def _run_plan(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        p = rsa.tree_plan(s.parent, s.cu, s.kv_len, s.tree, pos0=100)
        return {"positions": p.positions, "mask": p.mask}
    cu, n = s.cu.long(), s.tree
    m = _closure(s.parent, cu, n)
    t = torch.arange(s.parent.numel(), device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    live = r < s.R
    r.clamp_(max=s.R - 1)
    i = (t - cu[r]).clamp_(max=n - 1)
    depth = m.sum(2).long() - 1
    base = s.kv_len.long() - (cu[1:] - cu[:-1])
    return {"positions": torch.where(live, 100 + base[r] + depth[r, i], 0), "mask": _packed(m, r, i, _pages(n, 32)) * live[:, None]}


def _dense(cache, pages):
    """Keys of page lists [..., n] as [..., Hkv, n * page, d] in 32 bits."""
    x = cache[pages.clamp(min=0).long()].float()
    x = x.movedim(-3, -4)  # [..., Hkv, n, page, d]
    return x.flatten(-3, -2)


def _run_attn(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        out, lse = rsa.tree_attn(s.q, s.cache_k, s.cache_v, s.cu, s.table, s.kv_len, s.mask, prefix_pages=s.prefix_pages, prefix_len=s.prefix)
        return {"out": out, "lse": lse}
    R, n, Hkv, d = s.R, s.most, s.Hkv, s.d
    G = s.Hq // Hkv
    scale = 1 / math.sqrt(d)
    q = torch.zeros(R, n, s.Hq, d, device="cuda")
    q[s.r, s.i] = s.q.float()
    q = q.view(R, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, d)
    used = _pages(s.longest, s.page)
    k, v = _dense(s.cache_k, s.table[:, :used]), _dense(s.cache_v, s.table[:, :used])  # [R, Hkv, L, d]
    key = torch.arange(k.shape[2], device="cuda")
    cu = s.cu.long()
    base = s.kv_len.long() - (cu[1:] - cu[:-1])
    j = key - base[:, None]  # the drafted token that a key belongs to
    word = torch.zeros(R, n, s.mask.shape[1], dtype=torch.int64, device="cuda")
    word[s.r, s.i] = s.mask.long()
    at = j.clamp(0, n - 1)[:, None, :].expand(R, n, -1)
    bit = word.gather(2, at // 32) >> (at % 32) & 1
    seen = (j < 0)[:, None] | ((j < n)[:, None] & (bit > 0))  # [R, n, L]
    sc = ((q @ k.transpose(2, 3)) * scale).view(R, Hkv, n, G, -1)
    sc = torch.where(seen[:, None, :, None, :], sc, -math.inf).view(R, Hkv, n * G, -1)
    m = sc.amax(-1)
    if s.prefix:
        kp, vp = _dense(s.cache_k, s.prefix_pages)[:, : s.prefix], _dense(s.cache_v, s.prefix_pages)[:, : s.prefix]  # [Hkv, P, d]
        sp = (q @ kp.transpose(1, 2)) * scale
        m = torch.maximum(m, sp.amax(-1))
        ep = torch.exp(sp - m[..., None])
    e = torch.exp(sc - m[..., None])
    l, o = e.sum(-1), e @ v
    if s.prefix:
        l, o = l + ep.sum(-1), o + ep @ vp
    o, lse = o / l[..., None], m + torch.log(l)
    o = o.view(R, Hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(R, n, s.Hq, d)[s.r, s.i]
    lse = lse.view(R, Hkv, n, G).permute(0, 2, 1, 3).reshape(R, n, s.Hq)[s.r, s.i]
    return {"out": o.to(s.q.dtype), "lse": lse}


def _run_compact(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        new_len = rsa.cache_compact(s.cache_k, s.cache_v, s.table, s.base, s.kv_len, s.lists, s.keep_len)
        return {"k_cache": s.cache_k, "v_cache": s.cache_v, "kv_len": new_len}
    page, i = s.page, torch.arange(s.lists.shape[1], device="cuda")
    to = s.base.long()[:, None] + i
    source = s.base.long()[:, None] + s.lists.long()
    moved = (i < s.keep_len[:, None]) & (source != to)
    r = torch.arange(s.R, device="cuda")[:, None].expand_as(to)[moved]
    source, to = source[moved], to[moved]
    ps, pt = s.table[r, source // page].long(), s.table[r, to // page].long()
    for c in (s.cache_k, s.cache_v):
        c[:, pt, :, to % page] = c[:, ps, :, source % page]
    return {"k_cache": s.cache_k, "v_cache": s.cache_v, "kv_len": s.base + s.keep_len}


def _give_back(s):
    """The plain form of freeing: (free start, pages freed, entries given back)."""
    col = torch.arange(s.table.shape[1], device="cuda")
    gone = (col >= ((s.keep_len + s.page - 1) // s.page)[:, None]) & (col < ((s.kv_len + s.page - 1) // s.page)[:, None])
    at = torch.where(gone, s.table.long(), s.n_pages).flatten()
    count = torch.zeros(s.n_pages + 1, dtype=torch.int32, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:-1]
    shares = s.shares if "shares" in s else torch.zeros_like(count)
    freed = count > shares
    if "shares" in s:
        s.shares.copy_(torch.where(freed, 0, shares - count))
    n = freed.sum()
    start = s.free_start[0] - n
    place = start + torch.cumsum(freed, 0) - 1
    page = torch.arange(s.n_pages, device="cuda", dtype=torch.int32)
    pool = torch.cat([s.free, s.free[:1]])  # (the last entry takes what is not freed)
    pool[torch.where(freed, place, s.free.numel())] = page
    s.free.copy_(pool[:-1])
    return start, n, gone.sum()


def _run_free(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        info = rsa.page_free(s.table, s.kv_len, s.keep_len, s.free, s.free_start, s.page, s.n_pages)
        return {"free": s.free, "info": info}
    start, n, gone = _give_back(s)
    return {"free": s.free, "info": torch.stack([torch.zeros_like(n), n, gone, start])}


def _run_beam(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        freed = rsa.page_free(s.table, s.kv_len, s.keep_len, s.free, s.free_start, s.page, s.n_pages, shares=s.shares)
        info = rsa.page_fork(s.cache_k, s.cache_v, s.table, s.kv_len, s.src, s.dst, s.free, free_start=freed[3:], shares=s.shares)
    else:
        start, n, gone = _give_back(s)
        freed = torch.stack([torch.zeros_like(n), n, gone, start])
        src, dst = s.src.long(), s.dst.long()
        lens = s.kv_len[src].long()
        full, rest = lens // s.page, lens % s.page
        need = rest > 0
        place = start + torch.cumsum(need, 0) - 1
        col = torch.arange(s.table.shape[1], device="cuda")
        shared = col < full[:, None]
        old = s.table[src]
        last = old.gather(1, full[:, None])[:, 0].clamp(min=0).long()
        fresh = s.free[place.clamp(0, s.free.numel() - 1)]
        row = torch.where(shared, old, s.table[dst])
        s.table[dst] = torch.where((col == full[:, None]) & need[:, None], fresh[:, None], row)
        at = torch.where(shared, old.long(), s.n_pages).flatten()
        s.shares += torch.zeros(s.n_pages + 1, dtype=torch.int32, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:-1]
        s.kv_len[dst] = s.kv_len[src]
        f, line = (torch.arange(s.page, device="cuda") < rest[:, None]).nonzero(as_tuple=True)
        for c in (s.cache_k, s.cache_v):
            c[:, fresh[f].long(), :, line] = c[:, last[f], :, line]
        info = torch.stack([torch.zeros_like(n), shared.sum(), need.sum(), start + need.sum()])
    return {"table": s.table, "kv_len": s.kv_len, "shares": s.shares, "free": s.free, "k_cache": s.cache_k, "v_cache": s.cache_v,
            "freed": freed, "info": info}


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    op, R = case["op"], case["R"]
    size = 4 if case.get("dtype") == F32 else 2
    if op == "plan":
        T = sum(_tree_sizes(case)) + case["pad"]
        return {"bytes": T * 12 + R * 8 + T * 4 * _pages(case["tree"], 32), "flops": 0}
    if op == "attn":
        sizes, cached = _tree_sizes(case), _attn_lens(case)
        T, Hq, Hkv, d, w = sum(sizes), case["Hq"], case["Hkv"], case["d"], case["width"]
        keys = case["prefix"] + sum(cached) + T
        # a token of index i has some 2 i / (width + 1) ancestors
        pairs = T * case["prefix"] + sum(n * c + n + n * (n - 1) // (w + 1) for n, c in zip(sizes, cached))
        return {"bytes": keys * Hkv * 2 * d * size + T * Hq * (2 * d * size + 4) + T * 4 * _pages(max(sizes), 32) + _pages(keys, case["page"]) * 4,
                "flops": 4 * d * Hq * pairs}
    if op == "free":
        lens, keep = _free_lens(case)
        gone = sum(_pages(n, case["page"]) - _pages(k, case["page"]) for n, k in zip(lens, keep))
        return {"bytes": 8 * gone + 8 * R, "flops": 0}
    row = case["layers"] * 2 * case["Hkv"] * case["d"] * size
    if op == "compact":
        _, _, kept = _compact_lens(case)
        stay = 4 * R if case["window"] else 0  # rows that stay where they are
        return {"bytes": 2 * row * (sum(kept) - stay) + 4 * sum(kept) + 16 * R, "flops": 0}
    lens, src, dst = _beam_plan(case)
    page = case["page"]
    entries = sum(_pages(lens[r], page) for r in src)
    # each source's partial page is read once, whatever the number of its forks
    return {"bytes": row * (sum(lens[r] % page for r in src) + sum(lens[r] % page for r in set(src))) + entries * 16, "flops": 0}


# ---- the operators' definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("plan", "free"):
        return None  # whole numbers throughout
    if op == "attn":
        return _exact_attn(s)
    page, kc, vc = s.page, s.cache_k.double(), s.cache_v.double()
    if op == "compact":
        table = s.table.tolist()
        lists, base, kept = s.lists.tolist(), s.base.tolist(), s.keep_len.tolist()
        old = (kc.clone(), vc.clone())
        for r in range(s.R):
            at = [(base[r] + i, base[r] + lists[r][i]) for i in range(kept[r]) if lists[r][i] != i]
            where = lambda side: (torch.tensor([table[r][p[side] // page] for p in at], dtype=torch.int64, device="cuda"),  # noqa: E731
                                  torch.tensor([p[side] % page for p in at], dtype=torch.int64, device="cuda"))
            (pt, lt), (ps, ls) = where(0), where(1)
            for new, was in zip((kc, vc), old):
                new[:, pt, :, lt] = was[:, ps, :, ls]
        return {"k_cache": kc, "v_cache": vc, "kv_len": None}
    table, lens = s.table.tolist(), s.kv_len.tolist()
    for a, b in zip(s.src.tolist(), s.dst.tolist()):  # (the pages that the step before took are freed and taken again)
        at, n = lens[a] // page, lens[a] % page
        if n:
            for c in (kc, vc):
                c[:, table[b][at], :, :n] = c[:, table[a][at], :, :n]
    return {"table": None, "kv_len": None, "shares": None, "free": None, "k_cache": kc, "v_cache": vc, "freed": None, "info": None}


def _exact_attn(s):
    """One request and key head after the other."""
    T, G = s.q.shape[0], s.Hq // s.Hkv
    out = torch.zeros(T, s.Hq, s.d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, s.Hq, dtype=torch.float64, device="cuda")
    cu, lens = s.cu.tolist(), s.kv_len.tolist()
    rows = lambda c, pages, h, n: c[pages.long(), h].double().reshape(-1, s.d)[:n]  # noqa: E731
    for r in range(s.R):
        a, n = cu[r], cu[r + 1] - cu[r]
        pages = s.table[r, : _pages(lens[r], s.page)]
        word = s.mask[a:a + n].long() & 0xFFFFFFFF
        sees = torch.ones(n, s.prefix + lens[r], dtype=torch.bool, device="cuda")
        j = torch.arange(n, device="cuda")
        sees[:, s.prefix + lens[r] - n:] = (word[:, j // 32] >> (j % 32)) % 2 == 1
        for h in range(s.Hkv):
            k = torch.cat([rows(s.cache_k, s.prefix_pages, h, s.prefix), rows(s.cache_k, pages, h, lens[r])])
            v = torch.cat([rows(s.cache_v, s.prefix_pages, h, s.prefix), rows(s.cache_v, pages, h, lens[r])])
            x = s.q[a:a + n, h * G:(h + 1) * G].double()  # [n, G, d]
            sc = (x @ k.T / math.sqrt(s.d)).masked_fill(~sees[:, None], -math.inf)
            z = torch.logsumexp(sc, -1, keepdim=True)
            out[a:a + n, h * G:(h + 1) * G] = torch.exp(sc - z) @ v
            lse[a:a + n, h * G:(h + 1) * G] = z[..., 0]
    return {"out": out, "lse": lse}
