"""The serving operators next to the attention of this library, as cases to be measured.

Three operators that a decode step with a paged KV cache runs one after the other:

  plan     page_plan: block tables, slot map and positions of a step, from the requests' lengths
  rope     qk_norm_rope: RMS norm of every query and key head, the position rotation in the same
           pass, keys and values written to their cache slots; ropeb is its backward pass
  attn     prefix_attn: attention of every request's newest tokens over one shared prefix and the
           request's own paged keys

`own` False: plain torch, 32 bits (64 where angles or offsets need it), rounded once at the end.
`own` True: the package's calls.
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
        # one decode step of eight sequences (the batch of the page-1 shape), one token each
        {"name": "plan_decode_8", "op": "plan", "R": 8, "page": 64, "new": 1, "cached": 32768, "pad": 0},
        # a busy server: 4000 requests, prompts and single tokens mixed, batch padded
        {"name": "plan_mixed_4000", "op": "plan", "R": 4000, "page": 16, "new": 1000, "cached": 4000, "pad": 1000},
        # ---- rope -----------------------------------------------------------------------------
        # one decode step of 64 requests, 64 query heads over 8 key heads, batch padded by 7 rows
        {"name": "rope_decode_64", "op": "rope", "dtype": BF16, "T": 64, "pad": 7, "Hq": 64, "Hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "axes": 1, "page": 64, "cache": True},
        # a 32768-token prompt (the page-1 sequence), heads cut from one packed projection
        {"name": "rope_prompt_32768", "op": "rope", "dtype": BF16, "T": 32768, "pad": 0, "Hq": 64, "Hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "axes": 1, "page": 64, "cache": True},
        # video tokens in 32 bits: time, height and width turn interleaved pairs of small heads, an odd count
        {"name": "rope_video_f32", "op": "rope", "dtype": F32, "T": 10007, "pad": 0, "Hq": 16, "Hkv": 4, "d": 64, "rot": 48,
         "interleaved": True, "axes": 3, "page": 16, "cache": False},
        # the backward pass of a training step: 64 query heads over 8 key heads, 8192 tokens (a ring chunk)
        {"name": "ropeb_chunk_8192", "op": "ropeb", "dtype": BF16, "T": 8192, "pad": 0, "Hq": 64, "Hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "axes": 1, "page": 64, "cache": False},
        # the same in 32 bits at small heads and an odd length
        {"name": "ropeb_f32_1001", "op": "ropeb", "dtype": F32, "T": 1001, "pad": 0, "Hq": 8, "Hkv": 8, "d": 64, "rot": 64,
         "interleaved": True, "axes": 1, "page": 64, "cache": False},
        # ---- attn -----------------------------------------------------------------------------
        # one request, no prefix, a short context: latency alone
        {"name": "attn_one_1000", "op": "attn", "dtype": BF16, "R": 1, "new": 1, "Hq": 64, "Hkv": 8, "d": 128, "page": 64,
         "prefix": 0, "own_lo": 1000, "own_hi": 1000},
        # 64 requests behind a 32768-token document, own keys from a few to 2000
        {"name": "attn_prefix_32768", "op": "attn", "dtype": BF16, "R": 64, "new": 1, "Hq": 64, "Hkv": 8, "d": 128, "page": 64,
         "prefix": 32768, "own_lo": 4, "own_hi": 2000},
        # plain heads (as many key heads as query heads), four tokens a request, 100000 shared tokens, small pages
        {"name": "attn_heads32_100000", "op": "attn", "dtype": BF16, "R": 8, "new": 4, "Hq": 32, "Hkv": 32, "d": 128, "page": 16,
         "prefix": 100000, "own_lo": 4, "own_hi": 1000},
        # no shared prefix, four long contexts of their own: a plain paged decode bound by the cache
        {"name": "attn_long_262144", "op": "attn", "dtype": BF16, "R": 4, "new": 1, "Hq": 64, "Hkv": 8, "d": 128, "page": 128,
         "prefix": 0, "own_lo": 131072, "own_hi": 262144},
        # 32 bits, small heads, an odd prefix
        {"name": "attn_f32_4097", "op": "attn", "dtype": F32, "R": 5, "new": 2, "Hq": 8, "Hkv": 4, "d": 64, "page": 32,
         "prefix": 4097, "own_lo": 2, "own_hi": 500},
    ]


# What a drawn case may cost at most: the largest listed one's bytes and operations.
_MOST = {}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["plan", "rope", "ropeb", "attn", "attn"])
    if op == "plan":
        return {"op": op, "R": _log(rng, 1, 4000), "page": rng.choice([16, 32, 64, 128]), "new": _log(rng, 1, 1000),
                "cached": _log(rng, 1, 40000), "pad": rng.randrange(0, 500)}
    dtype = rng.choice([BF16, BF16, F32])
    d = rng.choice([64, 128])
    G, Hkv = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    if op in ("rope", "ropeb"):
        rot = rng.choice([d, d, 32, 48])
        return {"op": op, "dtype": dtype, "T": _log(rng, 1, 32768 if op == "rope" else 8192), "pad": 0 if op == "ropeb" else rng.choice([0, 3]),
                "Hq": G * Hkv, "Hkv": Hkv, "d": d, "rot": rot, "interleaved": rng.random() < 0.4, "axes": rng.choice([1, 1, 2, 3]),
                "page": rng.choice([16, 32, 64, 128]), "cache": op == "rope" and rng.random() < 0.6}
    new = rng.choice([1, 1, 1, 2, 5])
    small = dtype == F32  # the 32-bit path is for short contexts
    hi = _log(rng, new, 1000 if small else 100000)
    return {"op": op, "dtype": dtype, "R": _log(rng, 1, 16 if small else 100), "new": new, "Hq": G * Hkv, "Hkv": Hkv, "d": d,
            "page": rng.choice([16, 32, 64, 128]), "prefix": rng.choice([0, 1]) * _log(rng, 1, 8000 if small else 100000),
            "own_lo": max(new, hi // 8), "own_hi": hi}


def draw(rng):
    if not _MOST:
        for c in listed():
            w = work(c)
            m = _MOST.setdefault((c["op"], c.get("dtype")), {"bytes": 0, "flops": 0, "plain": 0})
            for k in ("bytes", "flops"):
                m[k] = max(m[k], w[k])
            if c["op"] == "attn":
                m["plain"] = max(m["plain"], _plain_keys(c))
    while True:
        c = _drawn(rng)
        m, w = _MOST[(c["op"], c.get("dtype"))], work(c)
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and (c["op"] != "attn" or _plain_keys(c) <= m["plain"]):
            return c


# ---- lengths: plain numbers that follow from the case alone -----------------------------------------


def _plan_lens(case):
    r = random.Random("plan %(R)d %(new)d %(cached)d" % case)
    new = [1 if case["new"] == 1 or r.random() < 0.8 else r.randint(1, case["new"]) for _ in range(case["R"])]
    old = [r.randint(0, case["cached"]) for _ in range(case["R"])]
    return old, new


def _attn_lens(case):
    r = random.Random("attn %(R)d %(own_lo)d %(own_hi)d" % case)
    lo, hi = math.log(case["own_lo"]), math.log(case["own_hi"])
    lens = [max(case["new"], int(round(math.exp(r.uniform(lo, hi))))) for _ in range(case["R"])]
    lens[0] = case["own_hi"]
    return lens


def _plain_keys(case):
    """Scores of the plain form, whose own keys are padded to the longest request's."""
    return case["R"] * case["new"] * case["Hq"] * (case["prefix"] + case["own_hi"])


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
    if case["op"] == "plan":
        return _prepare_plan(case, s, g)
    if case["op"] == "attn":
        return _prepare_attn(case, s, g)
    return _prepare_rope(case, s, g)


def _prepare_plan(case, s, g):
    old, new = _plan_lens(case)
    page = case["page"]
    have = [_pages(o, page) for o in old]
    need = [_pages(o + n, page) - h for o, n, h in zip(old, new, have)]
    s.max_pages = max(h + n for h, n in zip(have, need)) + 2
    s.n_pages = sum(have) + sum(need) + 100
    s.max_tokens = sum(new) + case["pad"]
    s.start = 7
    ids = torch.randperm(s.n_pages, generator=g, device="cuda", dtype=torch.int32)
    at = torch.zeros(case["R"], dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(have), 0)[:-1]
    at, hv = at.cuda(), torch.tensor(have, device="cuda")
    col = torch.arange(s.max_pages, device="cuda")
    table = torch.where(col < hv[:, None], ids[(at[:, None] + col).clamp_(max=s.n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    s.table = table.to(torch.int32).contiguous()
    # the pool of free pages, consumed from `start` on
    s.free = torch.cat([ids[sum(have):sum(have) + s.start].flip(0), ids[sum(have):]])[: s.start + sum(need) + 50].contiguous()
    s.free_start = torch.tensor([s.start], dtype=torch.int64, device="cuda")
    s.cached_len, s.new_len = _i32(old), _i32(new)
    return s


def _table(case):
    """cos and sin of every position's angles, taken in 64 bits."""
    half = case["rot"] // 2
    n = case["T"] + case["pad"] + 1000
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _sections(case):
    half, axes = case["rot"] // 2, case["axes"]
    first = half // axes
    return None if axes == 1 else [half - first * (axes - 1)] + [first] * (axes - 1)


def _prepare_rope(case, s, g):
    T, Hq, Hkv, d, dt = case["T"] + case["pad"], case["Hq"], case["Hkv"], case["d"], _dt(case)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    qkv = torch.empty(T, (Hq + 2 * Hkv) * d, dtype=dt, device="cuda")  # the packed projection that q, k and v are cut from
    qkv.copy_(randn(T, (Hq + 2 * Hkv) * d))
    s.q = qkv[:, : Hq * d].view(T, Hq, d)
    s.k = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    s.v = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    s.wq, s.wk = (1 + 0.1 * randn(d)).to(dt), (1 + 0.1 * randn(d)).to(dt)
    s.eps = 1e-6
    s.cos_sin = _table(case)
    far = s.cos_sin.shape[0]
    pos = torch.arange(T, device="cuda", dtype=torch.int64) + 500
    if case["axes"] > 1:
        pos = torch.randint(0, far, (case["axes"], T), generator=g, device="cuda", dtype=torch.int64)
    s.pos, s.sections = pos, _sections(case)
    if case["op"] == "ropeb":
        s.dq, s.dk = randn(T, Hq, d).to(dt), randn(T, Hkv, d).to(dt)
    s.cache_k = s.cache_v = s.slots = None
    if case["cache"]:
        page = case["page"]
        n_pages = _pages(T, page) + 3
        shape = (n_pages, Hkv, page, d)
        s.cache_k, s.cache_v = randn(*shape).to(dt), randn(*shape).to(dt)
        ids = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64)
        t = torch.arange(T, device="cuda")
        s.slots = ids[t // page] * page + t % page
        if case["pad"]:
            s.slots[case["T"]:] = -1  # the padded rows of the batch have no slot
    return s


def _prepare_attn(case, s, g):
    R, Hq, Hkv, d, dt, page = case["R"], case["Hq"], case["Hkv"], case["d"], _dt(case), case["page"]
    lens = _attn_lens(case)
    T = R * case["new"]
    np_prefix = _pages(case["prefix"], page)
    counts = [_pages(n, page) for n in lens]
    n_pages = np_prefix + sum(counts) + 3
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda", dtype=dt)  # noqa: E731
    s.q = randn(T, Hq, d)
    s.cache_k, s.cache_v = randn(n_pages, Hkv, page, d), randn(n_pages, Hkv, page, d)
    ids = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    s.prefix_pages = ids[:np_prefix].contiguous()
    s.max_pages = max(counts) + 1
    at = torch.zeros(R, dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(counts), 0)[:-1]
    at = at.cuda() + np_prefix
    col = torch.arange(s.max_pages, device="cuda")
    s.table = torch.where(col < torch.tensor(counts, device="cuda")[:, None], ids[(at[:, None] + col).clamp_(max=n_pages - 1)],
                          torch.full((), -1, dtype=torch.int32, device="cuda")).to(torch.int32).contiguous()
    s.kv_len = _i32(lens)
    s.cu_q = torch.arange(R + 1, device="cuda", dtype=torch.int32) * case["new"]
    s.longest = max(lens)
    return s


# ---- one pass ---------------------------------------------------------------------------------------


def run(s):
    return {"plan": _run_plan, "rope": _run_rope, "ropeb": _run_ropeb, "attn": _run_attn}[s["op"]](s)


def _run_plan(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        p = rsa.page_plan(s.cached_len, s.new_len, s.table, s.free, s.page, s.n_pages, s.max_tokens, free_start=s.free_start, pos0=100)
        return {"table": s.table, "cu_new": p.cu_new, "kv_len": p.kv_len, "slot_map": p.slot_map, "positions": p.positions, "info": p.info}
    page, table = s.page, s.table
    c, n = s.cached_len.long(), s.new_len.long()
    have = (c + page - 1) // page
    need = (c + n + page - 1) // page - have
    ends, taken = torch.cumsum(n, 0), torch.cumsum(need, 0)
    start = s.free_start[0]
    bad = [((c < 0) | (n < 0)).any(), (have + need > table.shape[1]).any(), start + taken[-1] > s.free.numel(), ends[-1] > s.max_tokens]
    code = torch.where(bad[0], 1, torch.where(bad[1], 2, torch.where(bad[2], 3, torch.where(bad[3], 4, 0))))
    ok = code == 0
    col = torch.arange(table.shape[1], device="cuda")
    fresh = ok & (col >= have[:, None]) & (col < (have + need)[:, None])
    at = start + (taken - need)[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, s.free[at.clamp_(0, s.free.numel() - 1)], table))
    t = torch.arange(s.max_tokens, device="cuda")
    r = torch.searchsorted(ends, t, right=True).clamp_(max=c.numel() - 1)
    live = ok & (t < ends[-1])
    pos = c[r] + t - (ends - n)[r]
    slot = table[r, (pos // page).clamp_(0, table.shape[1] - 1)].long() * page + pos % page
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu = torch.cat([zero, ends]) * ok
    info = torch.stack([code, ends[-1] * ok, taken[-1] * ok, start + taken[-1] * ok])
    return {"table": table, "cu_new": cu.int(), "kv_len": (c + n * ok).int(), "slot_map": torch.where(live, slot, -1),
            "positions": torch.where(live, pos + 100, 0), "info": info}


def _angles(s):
    """cos and sin [T, 1, rot / 2] of every token, each frequency at its own axis' position."""
    half = s.rot // 2
    if s.sections is None:
        cs = s.cos_sin[s.pos]
    else:
        axis = torch.repeat_interleave(torch.arange(len(s.sections), device="cuda"), torch.tensor(s.sections, device="cuda"), output_size=half)
        f = torch.arange(half, device="cuda")
        p = s.pos[axis].t()  # [T, half]
        cs = torch.cat([s.cos_sin[p, f], s.cos_sin[p, f + half]], 1)
    return cs[:, None, :half], cs[:, None, half:]


def _pairs(s, x):
    half = s.rot // 2
    if s.interleaved:
        return x[..., 0:s.rot:2], x[..., 1:s.rot:2]
    return x[..., :half], x[..., half:s.rot]


def _join(s, a, b, rest):
    if s.interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_rotate(s, x, w, cos, sin):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s.eps) * w.float()
    a, b = _pairs(s, y)
    return _join(s, a * cos - b * sin, a * sin + b * cos, y[..., s.rot:])


def _run_rope(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        if s.cache:
            q, _ = rsa.qk_norm_rope(s.q, s.k, s.wq, s.wk, s.pos, s.cos_sin, eps=s.eps, interleaved=s.interleaved, sections=s.sections,
                                    v=s.v, slot_map=s.slots, k_cache=s.cache_k, v_cache=s.cache_v)
            return {"q": q, "k_cache": s.cache_k, "v_cache": s.cache_v}
        q, k = rsa.qk_norm_rope(s.q, s.k, s.wq, s.wk, s.pos, s.cos_sin, eps=s.eps, interleaved=s.interleaved, sections=s.sections)
        return {"q": q, "k": k}
    cos, sin = _angles(s)
    q = _norm_rotate(s, s.q, s.wq, cos, sin).to(s.q.dtype)
    k = _norm_rotate(s, s.k, s.wk, cos, sin).to(s.k.dtype)
    if not s.cache:
        return {"q": q, "k": k}
    live, slot, v = s.slots, s.slots, s.v
    if s.pad:
        live = s.slots >= 0
        slot, k, v = s.slots[live], k[live], v[live]
    s.cache_k[slot // s.page, :, slot % s.page] = k
    s.cache_v[slot // s.page, :, slot % s.page] = v
    return {"q": q, "k_cache": s.cache_k, "v_cache": s.cache_v}


def _norm_rotate_grad(s, dy, x, w, cos, sin):
    x, w, dy = x.float(), w.float(), dy.float()
    a, b = _pairs(s, dy)
    g = _join(s, a * cos + b * sin, b * cos - a * sin, dy[..., s.rot:])  # the rotation turned back
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s.eps)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


def _run_ropeb(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        dq, dk, dwq, dwk = rsa.qk_norm_rope_bwd(s.dq, s.dk, s.q, s.k, s.wq, s.wk, s.pos, s.cos_sin, eps=s.eps,
                                                interleaved=s.interleaved, sections=s.sections)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    cos, sin = _angles(s)
    dq, dwq = _norm_rotate_grad(s, s.dq, s.q, s.wq, cos, sin)
    dk, dwk = _norm_rotate_grad(s, s.dk, s.k, s.wk, cos, sin)
    return {"dq": dq.to(s.q.dtype), "dk": dk.to(s.k.dtype), "dwq": dwq, "dwk": dwk}


def _dense(cache, pages):
    """Keys of page lists [..., n] as [..., Hkv, n * page, d] in 32 bits."""
    x = cache[pages.clamp(min=0).long()].float()
    x = x.movedim(-3, -4)  # [..., Hkv, n, page, d]
    return x.flatten(-3, -2)


def _run_attn(s):
    if own:
        import context_attention_rsa_gb300 as rsa
        out, lse = rsa.prefix_attn(s.q, s.cache_k, s.cache_v, s.cu_q, s.table, s.kv_len, prefix_pages=s.prefix_pages, prefix_len=s.prefix)
        return {"out": out, "lse": lse}
    R, n, Hkv, d = s.R, s.new, s.Hkv, s.d
    G = s.Hq // Hkv
    scale = 1 / math.sqrt(d)
    q = s.q.float().view(R, n, Hkv, G, d)
    used = _pages(s.longest, s.page)
    k, v = _dense(s.cache_k, s.table[:, :used]), _dense(s.cache_v, s.table[:, :used])  # [R, Hkv, L, d]
    key = torch.arange(k.shape[2], device="cuda")
    seen = key < (s.kv_len.long()[:, None] - n + 1 + torch.arange(n, device="cuda"))[:, :, None]  # [R, n, L]
    sc = (q.permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, d) @ k.transpose(2, 3)) * scale
    sc = torch.where(seen[:, None, :, None, :], sc.view(R, Hkv, n, G, -1), -math.inf)  # [R, Hkv, n, G, L]
    m = sc.amax(-1)
    if s.prefix:
        kp, vp = _dense(s.cache_k, s.prefix_pages)[:, : s.prefix], _dense(s.cache_v, s.prefix_pages)[:, : s.prefix]  # [Hkv, P, d]
        sp = (q.permute(2, 0, 1, 3, 4).reshape(Hkv, R * n * G, d) @ kp.transpose(1, 2)) * scale
        mp = sp.amax(-1).view(Hkv, R, n, G).transpose(0, 1)
        m = torch.maximum(m, mp)
        ep = torch.exp(sp - m.transpose(0, 1).reshape(Hkv, R * n * G, 1))
        lp = ep.sum(-1).view(Hkv, R, n, G).transpose(0, 1)
        op = (ep @ vp).view(Hkv, R, n, G, d).transpose(0, 1)
    e = torch.exp(sc - m[..., None])
    l = e.sum(-1)
    o = (e.view(R, Hkv, n * G, -1) @ v).view(R, Hkv, n, G, d)
    if s.prefix:
        l, o = l + lp, o + op
    o = (o / l[..., None]).permute(0, 2, 1, 3, 4).reshape(R * n, s.Hq, d)
    lse = (m + torch.log(l)).permute(0, 2, 1, 3).reshape(R * n, s.Hq)
    return {"out": o.to(s.q.dtype), "lse": lse}


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _plan_lens(case)
        page, tokens = case["page"], sum(new) + case["pad"]
        fresh = sum(_pages(o + n, page) - _pages(o, page) for o, n in zip(old, new))
        partly = sum(1 for o in old if o % page)
        # lengths read, kv_len and cu_new written, new table entries read and written, half-full pages looked up, 16 bytes a token
        return {"bytes": 16 * case["R"] + 8 * fresh + 4 * partly + 16 * tokens, "flops": 0}
    size = 4 if case["dtype"] == F32 else 2
    if op == "attn":
        T, lens = case["R"] * case["new"], _attn_lens(case)
        keys = case["prefix"] + sum(lens)
        pairs = T * case["prefix"] + sum(case["new"] * n - case["new"] * (case["new"] - 1) // 2 for n in lens)
        return {"bytes": 2 * size * keys * case["Hkv"] * case["d"] + 2 * size * T * case["Hq"] * case["d"] + 4 * T * case["Hq"],
                "flops": 4 * pairs * case["Hq"] * case["d"]}
    T, d = case["T"] + case["pad"], case["d"]
    table = 4 * case["rot"] * T + 8 * case["axes"] * T
    if op == "ropeb":
        return {"bytes": 3 * size * T * (case["Hq"] + case["Hkv"]) * d + table, "flops": 20 * T * (case["Hq"] + case["Hkv"]) * d}
    moved = T * case["Hq"] + case["T"] * case["Hkv"] * (2 if case["cache"] else 1) + (0 if case["cache"] else case["pad"] * case["Hkv"])
    return {"bytes": 2 * size * moved * d + table + (8 * T if case["cache"] else 0), "flops": 10 * T * (case["Hq"] + case["Hkv"]) * d}


# ---- the definitions, in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers: the plain form's own are the answer
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    return _exact_rope(s)


def _exact_attn(s):
    out = torch.empty(s.R * s.new, s.Hq, s.d, dtype=torch.float64, device="cuda")
    lse = torch.empty(s.R * s.new, s.Hq, dtype=torch.float64, device="cuda")
    lens = _attn_lens(s)
    G = s.Hq // s.Hkv

    def rows(cache, pages, h, n):
        return cache[:, h][pages.long()].reshape(-1, s.d)[:n].double()

    for h in range(s.Hkv):
        kp, vp = (rows(c, s.prefix_pages, h, s.prefix) for c in (s.cache_k, s.cache_v))
        for r in range(s.R):
            pages = s.table[r, : _pages(lens[r], s.page)]
            k = torch.cat([kp, rows(s.cache_k, pages, h, lens[r])])
            v = torch.cat([vp, rows(s.cache_v, pages, h, lens[r])])
            for i in range(s.new):
                n = s.prefix + lens[r] - s.new + 1 + i  # what token i of the request sees
                x = s.q[r * s.new + i, h * G:(h + 1) * G].double()
                z = torch.logsumexp(x @ k[:n].T / math.sqrt(s.d), 1, keepdim=True)
                out[r * s.new + i, h * G:(h + 1) * G] = torch.exp(x @ k[:n].T / math.sqrt(s.d) - z) @ v[:n]
                lse[r * s.new + i, h * G:(h + 1) * G] = z[:, 0]
    return {"out": out, "lse": lse}


def _exact_rope(s):
    """The rotation as a product of complex numbers, the norm as a division; gradients by automatic differentiation."""
    half = s.rot // 2
    table = s.cos_sin.double()
    if s.sections is None:
        turn = torch.complex(table[:, :half], table[:, half:])[s.pos]
    else:
        parts, at = [], 0
        for axis, n in enumerate(s.sections):
            row = table[s.pos[axis]]
            parts.append(torch.complex(row[:, at:at + n], row[:, half + at:half + at + n]))
            at += n
        turn = torch.cat(parts, 1)

    def f(x, w):
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / s.d + s.eps) * w
        head, rest = y[..., : s.rot], y[..., s.rot:]
        if s.interleaved:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * turn[:, None]
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn[:, None]
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, rest], -1)

    names = (("q", s.q, s.wq), ("k", s.k, s.wk))
    if s.op == "ropeb":
        got = {}
        for name, x, w in names:
            x, w = x.double().requires_grad_(), w.double().requires_grad_()
            dx, dw = torch.autograd.grad(f(x, w), (x, w), s["d" + name].double())
            got["d" + name], got["dw" + name] = dx, dw
        return got
    q, k = (f(x.double(), w.double()) for _, x, w in names)
    if not s.cache:
        return {"q": q, "k": k}
    n = s.T  # rows before the padding
    kc, vc = s.cache_k.double(), s.cache_v.double()
    kc[s.slots[:n] // s.page, :, s.slots[:n] % s.page] = k[:n]
    vc[s.slots[:n] // s.page, :, s.slots[:n] % s.page] = s.v[:n].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}
