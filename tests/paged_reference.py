"""Plain 64-bit forms (numpy) of the operators over a paged KV cache, for the
tests, with the error bounds that the kernels' arithmetic implies.  Nothing
here shares code with the library."""
import numpy as np
import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16


def half_step(dtype):
    """Relative error of one rounding to `dtype`, at most."""
    return torch.finfo(dtype).eps / 2


def to64(t):
    return t.detach().to(torch.float64).cpu().numpy()


# ---- the step's plan -------------------------------------------------------------------


def page_plan(cached, new, table, free, page, max_tokens, start=0, pos0=0):
    """(table, cu_new, kv_len, slot_map, positions, info) by a plain loop over requests and tokens."""
    R, max_pages = table.shape
    table = table.copy()
    have = [-(-c // page) if c >= 0 else 0 for c in cached]
    total = [-(-(c + n) // page) if c >= 0 and n >= 0 else 0 for c, n in zip(cached, new)]
    taken = sum(t - h for h, t in zip(have, total))
    tokens = sum(max(n, 0) for n in new)
    code = 0
    if min(cached) < 0 or min(new) < 0:
        code = 1
    elif max(total) > max_pages:
        code = 2
    elif start < 0 or start + taken > len(free):
        code = 3
    elif tokens > max_tokens:
        code = 4
    slots, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    if code:
        return table, np.zeros(R + 1, np.int32), np.array(cached, np.int32), slots, pos, np.array([code, 0, 0, start])
    cu, at, row = [0], start, 0
    for r in range(R):
        for j in range(have[r], total[r]):
            table[r, j] = free[at]
            at += 1
        for t in range(cached[r], cached[r] + new[r]):
            slots[row] = int(table[r, t // page]) * page + t % page
            pos[row] = pos0 + t
            row += 1
        cu.append(row)
    return (table, np.array(cu, np.int32), np.array([c + n for c, n in zip(cached, new)], np.int32), slots, pos,
            np.array([0, tokens, taken, at]))


# ---- norm and rotation ------------------------------------------------------------------


def _turn(y, cos, sin, rot, interleaved):
    y = y.copy()
    h = rot // 2
    a, b = (y[..., 0:rot:2].copy(), y[..., 1:rot:2].copy()) if interleaved else (y[..., :h].copy(), y[..., h:rot].copy())
    u, v = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, v
    else:
        y[..., :h], y[..., h:rot] = u, v
    return y


def _factors(positions, cos_sin, sections):
    """cos, sin [T, 1, rot/2] from positions [T] or [axes, T]."""
    half = cos_sin.shape[1] // 2
    pos = positions.reshape(-1, positions.shape[-1])
    axis = np.repeat(np.arange(len(sections)), sections) if sections is not None else np.zeros(half, np.int64)
    f = np.arange(half)
    p = pos[axis].T  # [T, half]
    return cos_sin[p, f][:, None], cos_sin[p, f + half][:, None]


def norm_rope(x, w, positions, cos_sin, eps, interleaved=False, sections=None):
    """x [T, H, d], w [d] or None: (y, bound): bound is the error of an fp32 evaluation, before the last rounding."""
    d = x.shape[-1]
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = n if w is None else n * w
    # sum of d squares in lanes of 4 or 8 and up to 5 shuffles, halved by the root; 1/sqrt of 2 ulp; two products;
    # the rotation's two products and sum: below 32 roundings of values of at most the row's largest, twice
    bound = 32 * U32 * 2 * np.abs(y).max(-1, keepdims=True)
    if cos_sin is not None and cos_sin.shape[1]:
        cos, sin = _factors(positions, cos_sin, sections)
        y = _turn(y, cos, sin, cos_sin.shape[1], interleaved)
    return y, bound + 0 * y


def norm_rope_bwd(dy, x, w, positions, cos_sin, eps, interleaved=False, sections=None):
    """(dx, dw, bound of dx, sum of |terms| of dw)."""
    d = x.shape[-1]
    g = dy
    if cos_sin is not None and cos_sin.shape[1]:
        cos, sin = _factors(positions, cos_sin, sections)
        g = _turn(dy, cos, -sin, cos_sin.shape[1], interleaved)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    c = g if w is None else g * w
    m = (c * n).mean(-1, keepdims=True)
    dx = r * (c - n * m)
    ww = np.ones(d) if w is None else np.abs(w)
    gmax = 2 * np.abs(dy).max(-1, keepdims=True)  # a turned element is at most |a| + |b|
    cmax = gmax * ww.max()
    # as above, the mean's terms with their own roundings: below 64 of either term's size
    bound = 64 * U32 * r * (cmax + np.abs(n).max(-1, keepdims=True) * (np.abs(n) * cmax).mean(-1, keepdims=True))
    size = (gmax * np.abs(n)).sum((0, 1))
    return dx, (g * n).sum((0, 1)), bound + 0 * dx, size


# ---- attention --------------------------------------------------------------------------


def rows_of(cache, pages, head, n, page):
    """Rows [0, n) of one key head, through its page list."""
    idx = np.arange(n)
    return cache[pages[idx // page], head, idx % page]


def prefix_attn(q, kc, vc, cu, table, kv_len, prefix_pages, prefix_len):
    """(out, lse, out of |v|, largest |q||k| sum, keys): rows behind the last request are NaN."""
    T, Hq, d = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out, mag = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, size, keys = np.full((T, Hq), np.nan), np.full((T, Hq), 0.0), np.zeros((T, Hq))
    for r in range(len(kv_len)):
        n = cu[r + 1] - cu[r]
        if n <= 0:
            continue
        for h in range(Hkv):
            parts = [(rows_of(c, prefix_pages, h, prefix_len, page) if prefix_len else np.zeros((0, d)),
                      rows_of(c, table[r], h, kv_len[r], page)) for c in (kc, vc)]
            k, v = (np.concatenate(p) for p in parts)
            for i in range(n):
                m = prefix_len + max(0, kv_len[r] - n + 1 + i)
                rows = slice(h * G, (h + 1) * G)
                x = q[cu[r] + i, rows]
                if m == 0:
                    out[cu[r] + i, rows], mag[cu[r] + i, rows], lse[cu[r] + i, rows] = 0, 0, -np.inf
                    continue
                s = x @ k[:m].T / np.sqrt(d)
                top = s.max(-1, keepdims=True)
                e = np.exp(s - top)
                l = e.sum(-1, keepdims=True)
                out[cu[r] + i, rows] = e @ v[:m] / l
                mag[cu[r] + i, rows] = e @ np.abs(v[:m]) / l
                lse[cu[r] + i, rows] = (top + np.log(l))[:, 0]
                size[cu[r] + i, rows] = (np.abs(x) @ np.abs(k[:m]).T).max(-1) / np.sqrt(d)
                keys[cu[r] + i, rows] = m
    return out, lse, mag, size, keys


def assert_prefix_attn(out, lse, ref, dtype, T=None):
    """Compares a result with prefix_attn's, element by element, within what its arithmetic implies:
    a score is a sum of d products (relative to |q||k|), which moves every probability by as much; sums of `keys`
    terms; exp and log of a few steps; in bf16 the probabilities and the result rounded once each."""
    ro, rl, mag, size, keys = ref
    T = ro.shape[0] if T is None else T
    ro, rl, mag, size, keys = ro[:T], rl[:T], mag[:T], size[:T], keys[:T]
    o, l = to64(out)[:T], to64(lse)[:T]
    d = ro.shape[-1]
    fp = 2 * U32 if dtype == torch.bfloat16 else U32  # (tensor cores may cut instead of rounding)
    score = (d + 8) * fp * size
    rel = 2 * score + (keys + 64) * fp
    tol = rel[..., None] * mag + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + U16 * mag + U16 * np.abs(ro)
    else:
        tol = tol + U32 * np.abs(ro)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), empty)
    assert np.all(o[empty] == 0)
    assert np.isfinite(o).all()
    worst = (np.abs(o - ro) / tol).max(initial=0)
    assert worst <= 1, f"out is {worst:.3g} times its bound off"
    ltol = score + (keys + 64) * fp + 4 * U32 * np.abs(np.where(empty, 0, rl))
    fin = ~empty
    worst = (np.abs(l[fin] - rl[fin]) / ltol[fin]).max(initial=0)
    assert worst <= 1, f"lse is {worst:.3g} times its bound off"
