"""Plain 64-bit forms (numpy) of the calls for drafted tokens and the keeping of
pages, by loops over requests and tokens.  Nothing here shares code with the library."""
import numpy as np

import paged_reference as ref


def random_forest(rng, n, width):
    """Parents of n tokens, each one of the `width` tokens before it or none (-1)."""
    return [max(-1, i - 1 - int(rng.integers(0, width))) for i in range(n)]


def tree_plan(parent, cu, kv_len, words, T, pos0=0):
    """(positions [T], mask [T, words] as int32)."""
    pos, mask = np.zeros(T, np.int64), np.zeros((T, words), np.uint32)
    for r in range(len(kv_len)):
        n = cu[r + 1] - cu[r]
        for i in range(n):
            j, depth = i, 0
            while j >= 0:
                mask[cu[r] + i, j // 32] |= np.uint32(1 << (j % 32))
                j = parent[cu[r] + j]
                depth += 1
            pos[cu[r] + i] = pos0 + kv_len[r] - n + depth - 1
    return pos, mask.view(np.int32)


def sees(mask, i, j):
    """Whether the row's mask (int32 words) lets token i see drafted token j."""
    w = np.asarray(mask).view(np.uint32)
    return j <= i and j < 32 * len(w) and bool(w[j // 32] >> np.uint32(j % 32) & np.uint32(1))


def tree_attn(q, kc, vc, cu, table, kv_len, mask, prefix_pages, prefix_len):
    """As paged_reference.prefix_attn, for its assert_prefix_attn."""
    T, Hq, d = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out, mag = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, size, keys = np.full((T, Hq), np.nan), np.full((T, Hq), 0.0), np.zeros((T, Hq))
    for r in range(len(kv_len)):
        n = cu[r + 1] - cu[r]
        base = kv_len[r] - n
        for i in range(n):
            at = [c for c in range(max(base, 0))] + [base + j for j in range(n) if base + j >= 0 and sees(mask[cu[r] + i], i, j)]
            at = np.array(at, np.int64)
            rows_at = cu[r] + i
            for h in range(Hkv):
                rows = slice(h * G, (h + 1) * G)
                parts = [(ref.rows_of(c, prefix_pages, h, prefix_len, page) if prefix_len else np.zeros((0, d)),
                          c[table[r][at // page], h, at % page]) for c in (kc, vc)]
                k, v = (np.concatenate(p) for p in parts)
                x = q[rows_at, rows]
                if not len(k):
                    out[rows_at, rows], mag[rows_at, rows], lse[rows_at, rows] = 0, 0, -np.inf
                    continue
                s = x @ k.T / np.sqrt(d)
                top = s.max(-1, keepdims=True)
                e = np.exp(s - top)
                l = e.sum(-1, keepdims=True)
                out[rows_at, rows] = e @ v / l
                mag[rows_at, rows] = e @ np.abs(v) / l
                lse[rows_at, rows] = (top + np.log(l))[:, 0]
                size[rows_at, rows] = (np.abs(x) @ np.abs(k).T).max(-1) / np.sqrt(d)
                keys[rows_at, rows] = len(k)
    return out, lse, mag, size, keys


def compact(caches, table, base, keep, keep_len, page):
    """New contents of the caches [L, n_pages, H, page, d] and the new lengths."""
    new = [c.copy() for c in caches]
    for r, n in enumerate(keep_len):
        for i in range(n):
            a, b = base[r] + keep[r][i], base[r] + i
            for c, old in zip(new, caches):
                c[:, table[r][b // page], :, b % page] = old[:, table[r][a // page], :, a % page]
    return new, [b + n for b, n in zip(base, keep_len)]


def fork(caches, table, kv_len, src, dst, free, start, shares, page):
    """(caches, table, kv_len, shares, info), shares None: every page is copied."""
    caches, table, kv_len = [c.copy() for c in caches], table.copy(), list(kv_len)
    shares = None if shares is None else shares.copy()
    n_pages, at, shared = caches[0].shape[1], start, 0
    pages = lambda n: -(-n // page)  # noqa: E731
    code = 0
    if any(not 0 <= r < len(kv_len) for r in (*src, *dst)) or len(set(dst)) < len(dst) or set(src) & set(dst):
        code = 5
    elif any(not 0 <= kv_len[a] <= table.shape[1] * page for a in src):
        code = 1
    else:
        need = sum((kv_len[a] % page > 0) if shares is not None else pages(kv_len[a]) for a in src)
        if start < 0 or start + need > len(free):
            code = 3
    if code:
        return caches, table, kv_len, shares, [code, 0, 0, start]
    for a, b in zip(src, dst):
        n = kv_len[a]
        for j in range(pages(n)):
            rows, was = min(page, n - j * page), table[a, j]
            if shares is not None and rows == page:
                table[b, j] = was
                shared += 1
                if 0 <= was < n_pages:
                    shares[was] += 1
                continue
            table[b, j] = free[at]
            at += 1
            for c in caches:
                c[:, table[b, j], :, :rows] = c[:, was, :, :rows]
        kv_len[b] = n
    return caches, table, kv_len, shares, [0, shared, at - start, at]


def free_pages(table, kv_len, keep_len, free, start, shares, page, n_pages):
    """(free, shares, info)."""
    free, shares = free.copy(), None if shares is None else shares.copy()
    pages = lambda n: -(-n // page)  # noqa: E731
    if any(not 0 <= k <= n <= table.shape[1] * page for n, k in zip(kv_len, keep_len)):
        return free, shares, [1, 0, 0, start]
    left = np.zeros(n_pages, np.int64) if shares is None else shares.astype(np.int64)
    gone, entries = set(), 0
    for r in range(len(kv_len)):
        for j in range(pages(keep_len[r]), pages(kv_len[r])):
            p = table[r, j]
            entries += 1
            if left[p] == 0:
                gone.add(int(p))
            left[p] -= 1
    if not len(gone) <= start <= len(free):
        return free, shares, [6, 0, 0, start]
    if shares is not None:
        shares[:] = left
        shares[sorted(gone)] = 0
    free[start - len(gone):start] = sorted(gone)
    return free, shares, [0, len(gone), entries, start - len(gone)]
