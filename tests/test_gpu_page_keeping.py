"""cache_compact, page_fork and page_free on the GPU against plain loops: rows and whole
numbers, equal in every bit."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
from test_gpu_index_data import reported

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731


class Keeper:
    """Caches of several layers whose elements are all different, and tables of shuffled pages."""

    def __init__(self, lens, page, dtype=BF, Hkv=2, d=64, layers=2, seed=0, extra=10, wide=1, start=4):
        rng = np.random.default_rng(seed)
        self.page, self.rng = page, rng
        counts = [-(-n // page) for n in lens]
        self.n_pages = sum(counts) + extra
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), max(counts + [1]) + wide), -(1 << 30), np.int32)
        at = 0
        for r, n in enumerate(counts):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.lens = list(lens)
        self.free = np.concatenate([ids[:start], ids[at:], ids[start:at]]).astype(np.int32)  # the pool; `extra` free ones from `start`
        self.start = start
        shape = (layers, self.n_pages, Hkv, page, d)
        # (bf16 holds any 16 bits; patterns of NaN among them would not compare: small whole numbers times powers of two)
        g = torch.Generator().manual_seed(seed)
        self.caches = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
        self.dev = [c.cuda() for c in self.caches]

    def plain(self):
        return [c.float().numpy() for c in self.caches]

    def assert_caches(self, want):
        for got, w in zip(self.dev, want):
            assert np.array_equal(got.float().cpu().numpy(), w)


# ---- cache_compact -------------------------------------------------------------------------

def kept(rng, n, m):
    return sorted(rng.choice(n, m, replace=False).tolist())


@pytest.mark.parametrize("dtype,Hkv,d,layers,page", [(BF, 2, 64, 2, 16), (BF, 3, 128, 1, 64), (F, 1, 64, 5, 32), (F, 2, 128, 2, 128),
                                                     (BF, 1, 64, 37, 16)])
@pytest.mark.parametrize("base,drafted,most", [
    ([5, 0, 17, 100, 31, 16], [1, 3, 9, 40, 0, 17], 9), ([0], [1], 1), ([63], [130], 130), ([0, 7], [700, 500], 333), ([1] * 70, [5] * 70, 3)])
def test_compact_matches_the_definition(dtype, Hkv, d, layers, page, base, drafted, most):
    need_cuda()
    k = Keeper([b + n for b, n in zip(base, drafted)], page, dtype, Hkv, d, layers)
    m = [int(k.rng.integers(0, min(most, n) + 1)) for n in drafted]
    m[-1] = min(most, drafted[-1])
    lists = [kept(k.rng, n, c) for n, c in zip(drafted, m)]
    keep = np.full((len(base), most + 2), 1 << 30, np.int32)  # (entries past keep_len are not looked at)
    for r, x in enumerate(lists):
        keep[r, :len(x)] = x
    want, lens = dr.compact(k.plain(), k.table, base, lists, m, page)
    got = rsa.cache_compact(*k.dev, i32(k.table), i32(base), i32(k.lens), i32(keep), i32(m))
    rsa.check_device_error()
    assert got.tolist() == lens
    k.assert_caches(want)


def test_compact_forms():
    need_cuda()
    k = Keeper([40, 90, 8], 16)
    base, m = [10, 50, 8], [20, 25, 0]
    lists = [kept(k.rng, 30, 20), list(range(25)), []]       # the second keeps its first tokens where they are
    keep = np.zeros((3, 25), np.int32)
    for r, x in enumerate(lists):
        keep[r, :len(x)] = x
    want, lens = dr.compact(k.plain(), k.table, base, lists, m, 16)
    # one layer's caches, strided lists and tables, an output given, another stream
    keep_dev = torch.full((3, 40), 7, dtype=torch.int32, device="cuda")
    keep_dev[:, 3:28] = i32(keep)
    table = torch.full((3, 99), 3, dtype=torch.int32, device="cuda")
    table[:, 5:5 + k.table.shape[1]] = i32(k.table)
    out, side = i32([9, 9, 9]), torch.cuda.Stream()
    torch.cuda.synchronize()
    for layer in range(2):
        got = rsa.cache_compact(k.dev[0][layer], k.dev[1][layer], table[:, 5:5 + k.table.shape[1]], i32(base), i32(k.lens), keep_dev[:, 3:28],
                                i32(m), out=out, stream=side)
        side.synchronize()
        assert got is out and out.tolist() == lens
    k.assert_caches(want)
    rsa.check_device_error()


def test_compact_leaves_a_request_whose_list_cannot_be_followed():
    need_cuda()
    page = 16
    base, drafted = [10, 20, 5], [30, 30, 30]
    good = [[0, 4, 7, 29], [3, 8, 20], [1, 2]]
    for what, site in (([8, 8, 20], 0x9b), ([9, 8, 20], 0x9b), ([-1, 8, 20], 0x9b), ([3, 8, 30], 0x9b), ([3, 8, 1 << 30], 0x9b), ("page", 0x9c),
                       ("far page", 0x9c), ("negative", 0x9a), ("too many", 0x9a), ("base", 0x9a), ("shrunk", 0x9a), ("beyond", 0x9a)):
        k = Keeper([b + n for b, n in zip(base, drafted)], page)
        lists, m, b, lens, table = [list(x) for x in good], [4, 3, 2], list(base), list(k.lens), k.table.copy()
        if isinstance(what, list):
            lists[1] = what
        elif what == "page":
            table[1, 1] = -7
        elif what == "far page":
            table[1, 2] = k.n_pages
        elif what in ("negative", "too many"):
            m[1] = -1 if what == "negative" else 6
        elif what == "base":
            b[1] = -1
        elif what == "shrunk":
            lens[1] = 19
        else:
            lens[1] = table.shape[1] * page + 1
        keep = np.zeros((3, 5), np.int32)
        for r, x in enumerate(lists):
            keep[r, :len(x)] = x
        want, _ = dr.compact(k.plain(), table, [base[0], 0, base[2]], [lists[0], [], lists[2]], [4, 0, 2], page)
        got = rsa.cache_compact(*k.dev, i32(table), i32(b), i32(lens), i32(keep), i32(m))
        assert f"site code 0x{site:02x}" in reported(), what
        assert got.tolist() == [14, b[1], 7], what
        k.assert_caches(want)


def test_compact_refusals():
    need_cuda()
    k = Keeper([40, 90], 16)
    args = [*k.dev, i32(k.table), i32([10, 10]), i32(k.lens), i32([[0, 1], [0, 1]]), i32([2, 2])]
    for at, bad in ((0, k.dev[0].half()), (0, k.dev[0][:, :-1]), (1, k.dev[1].float()), (0, k.dev[0][0, 0]), (0, k.dev[0].cpu()),
                    (1, k.dev[0]), (2, args[2].long()), (2, args[2][:1]), (3, args[3].long()), (3, args[3][:1]), (4, i32([[1, 2]])),
                    (5, args[5][:1]), (5, args[5].t()), (5, args[5][:, :0]), (6, i32([1, 2, 3])), (6, [1, 2])):
        a = list(args)
        a[at] = bad
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.cache_compact(*a)
    for bad in (i32([1]), args[3], args[4], i64([1, 2])):
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.cache_compact(*args, out=bad)
    k.assert_caches(k.plain())


# ---- page_fork -----------------------------------------------------------------------------

@pytest.mark.parametrize("shared", [True, False], ids=["shared", "copied"])
@pytest.mark.parametrize("dtype,Hkv,d,layers,page", [(BF, 2, 64, 2, 16), (BF, 5, 128, 1, 64), (F, 1, 128, 3, 32), (F, 2, 64, 1, 128)])
@pytest.mark.parametrize("lens,src,dst", [
    ([37, 0, 5], [0], [1]), ([64, 128, 1, 0], [0, 1], [2, 3]), ([300, 0, 0, 0, 17, 9], [0, 4, 0, 0], [1, 5, 3, 2]),
    ([0, 5], [0], [1]), ([33] * 40, [0, 1] * 19, list(range(2, 40))), ([1000, 0], [0], [1])])
def test_fork_matches_the_definition(lens, src, dst, dtype, Hkv, d, layers, page, shared):
    need_cuda()
    need = sum(-(-lens[a] // page) for a in src)
    k = Keeper(lens, page, dtype, Hkv, d, layers, extra=need + 3)
    k.table = np.pad(k.table, ((0, 0), (0, max(-(-n // page) for n in lens))), constant_values=-5)
    shares = k.rng.integers(0, 3, k.n_pages).astype(np.int32) if shared else None
    want = dr.fork(k.plain(), k.table, k.lens, src, dst, k.free, k.start, shares, page)
    table, kv, sh = i32(k.table), i32(k.lens), i32(shares) if shared else None
    info = rsa.page_fork(*k.dev, table, kv, i32(src), i32(dst), i32(k.free), free_start=i64([k.start]), shares=sh)
    rsa.check_device_error()
    assert info.tolist() == want[4] and want[4][0] == 0
    assert np.array_equal(table.cpu().numpy(), want[1]) and kv.tolist() == want[2]
    assert not shared or np.array_equal(sh.cpu().numpy(), want[3])
    k.assert_caches(want[0])


def test_forks_that_cannot_be_made_change_nothing():
    need_cuda()
    page = 16
    for src, dst, change, status in (
            ([0], [0], {}, 5), ([0, 1], [2, 2], {}, 5), ([0, 2], [2, 3], {}, 5), ([-1], [1], {}, 5), ([4], [1], {}, 5), ([0], [4], {}, 5),
            ([0], [-2147483648], {}, 5), ([1], [2], dict(kv=-1), 1), ([1], [2], dict(kv=1 << 30), 1), ([0, 0, 0], [1, 2, 3], dict(start=20), 3),
            ([0], [2], dict(start=-1), 3), ([0], [2], dict(start=1 << 40), 3)):
        for shared in (True, False):
            k = Keeper([40, 20, 9, 50], page, extra=15)
            if "kv" in change:
                k.lens[1] = change["kv"]
            start = change.get("start", k.start)
            shares = np.zeros(k.n_pages, np.int32) if shared else None
            table, kv, sh = i32(k.table), i32(k.lens), i32(shares) if shared else None
            pool = k.free[:k.start + 15 + 1] if "start" not in change else k.free[:21]
            want = dr.fork(k.plain(), k.table, k.lens, src, dst, pool, start, shares, page)
            info = rsa.page_fork(*k.dev, table, kv, i32(src), i32(dst), i32(pool), free_start=i64([start]), shares=sh)
            rsa.check_device_error()
            assert info.tolist() == want[4] and want[4][0] == (status if shared or status != 3 else 3), (src, dst, change)
            assert np.array_equal(table.cpu().numpy(), k.table) and kv.tolist() == k.lens
            assert not shared or (sh == 0).all()
            k.assert_caches(k.plain())


def test_fork_without_a_start_and_with_bad_pages():
    need_cuda()
    k = Keeper([40, 20, 9], 16)
    k.free[:2] = k.free[k.start:k.start + 2]
    table, kv, sh, info = i32(k.table), i32(k.lens), i32([0] * k.n_pages), i64([7, 7, 7, 7])
    want = dr.fork(k.plain(), k.table, k.lens, [0], [2], k.free, 0, np.zeros(k.n_pages, np.int32), 16)
    got = rsa.page_fork(*k.dev, table, kv, i32([0]), i32([2]), i32(k.free), shares=sh, out=info)
    assert got is info and info.tolist() == want[4] == [0, 2, 1, 1]
    k.assert_caches(want[0])
    # a full page that is none is handed on, not counted; a partial one or a fresh one that is none is not copied
    for row, at, value in ((0, 0, -3), (0, 2, k.n_pages), (None, k.start, 1 << 30)):
        k = Keeper([40, 20, 9], 16)
        if row is None:
            k.free[at] = value
        else:
            k.table[row, at] = value
        table, sh = i32(k.table), i32([0] * k.n_pages)
        info = rsa.page_fork(*k.dev, table, i32(k.lens), i32([0]), i32([2]), i32(k.free), free_start=i64([k.start]), shares=sh)
        assert f"site code 0x9d, first bad index {value})" in reported()
        assert info.tolist() == [0, 2, 1, k.start + 1]
        assert table[2, :3].tolist() == [*k.table[0, :2], k.free[k.start]]
        assert sh.sum() == (1 if (row, at) == (0, 0) else 2)
        if (row, at) != (0, 0):
            k.assert_caches(k.plain())


def test_most_requests_and_forks():
    need_cuda()
    R, F, page = 16384, 8000, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    n_pages = R - F + F
    kc, vc = (torch.randn(n_pages, 1, page, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    order = torch.randperm(R, generator=g, device="cuda")
    dst, rest = order[:F], order[F:]
    table = torch.full((R, 1), -1, dtype=torch.int32, device="cuda")
    table[rest, 0] = torch.arange(R - F, dtype=torch.int32, device="cuda")
    kv = torch.zeros(R, dtype=torch.int32, device="cuda")
    kv[rest] = torch.randint(1, page, (R - F,), generator=g, device="cuda", dtype=torch.int32)
    src = rest[torch.randint(0, R - F, (F,), generator=g, device="cuda")]
    free = torch.arange(R - F, n_pages, dtype=torch.int32, device="cuda").flip(0).contiguous()
    shares = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    was = kc.clone(), vc.clone()
    info = rsa.page_fork(kc, vc, table, kv, src.int(), dst.int(), free, shares=shares)
    rsa.check_device_error()
    assert info.tolist() == [0, 0, F, F] and not shares.any()
    assert torch.equal(kv[dst], kv[src]) and torch.equal(table[dst, 0], free)
    rows = torch.arange(page, device="cuda") < kv[dst][:, None]
    for c, w in zip((kc, vc), was):
        w[free.long()] = torch.where(rows[:, None, :, None], w[table[src, 0].long()], w[free.long()])
        assert torch.equal(c, w)
    with pytest.raises(rsa.RsaError):
        rsa.page_fork(kc, vc, table, kv, order[:8001].int(), order[:8001].int(), free)


@pytest.mark.parametrize("n_pages", [780000, 780001])
def test_most_requests_with_the_most_pages_that_fit(n_pages):
    # the two forms of the bitmap meet at 780000 pages; all of shared memory is in use there
    need_cuda()
    R = 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randperm(n_pages, generator=g, device="cuda")[:R * 40].int().view(R, 40).contiguous()
    kv = torch.randint(0, 641, (R,), generator=g, device="cuda", dtype=torch.int32)
    keep = (kv * torch.rand(R, generator=g, device="cuda")).int()
    col = torch.arange(40, device="cuda")
    gone = table[(col >= (keep[:, None] + 15) // 16) & (col < (kv[:, None] + 15) // 16)]
    for shares in (None, torch.zeros(n_pages, dtype=torch.int32, device="cuda")):
        free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        info = rsa.page_free(table, kv, keep, free, i64([n_pages]), 16, n_pages, shares=shares)
        rsa.check_device_error()
        n = gone.numel()
        assert info.tolist() == [0, n, n, n_pages - n]
        assert torch.equal(free[n_pages - n:], gone.sort().values) and (free[:n_pages - n] == -1).all()


def test_fork_refusals():
    need_cuda()
    k = Keeper([40, 20], 16)
    args = [*k.dev, i32(k.table), i32(k.lens), i32([0]), i32([1]), i32(k.free)]
    start, shares = i64([k.start]), i32([0] * k.n_pages)
    for at, bad in ((0, k.dev[1]), (1, k.dev[1][:1]), (2, args[2].long()), (3, args[3][:1]), (4, i32([0, 0])), (5, i64([1])), (4, i32([])),
                    (6, args[6].long()), (5, args[4])):
        a = list(args)
        a[at] = bad
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            info = rsa.page_fork(*a, free_start=start, shares=shares)
            if info[0] == 5:  # (dst is src: found on the device)
                raise ValueError
    for kw in (dict(shares=shares[:-1]), dict(shares=shares.long()), dict(free_start=start.int()), dict(free_start=start[:0]),
               dict(out=i64([1, 2, 3])), dict(out=i32([1, 2, 3, 4]))):
        with pytest.raises((ValueError, TypeError)):
            rsa.page_fork(*args, **{"free_start": start, "shares": shares, **kw})
    k.assert_caches(k.plain())


# ---- page_free -----------------------------------------------------------------------------

def free_case(lens, keep, page, shared, seed=0, sharing=None, extra=20):
    """Tables whose rows may share their first pages with row 0 (`sharing`: pages of it), and a pool with room."""
    k = Keeper(lens, page, layers=1, Hkv=1, seed=seed, extra=extra)
    shares = np.zeros(k.n_pages, np.int32)
    for r, n in (sharing or {}).items():
        k.table[r, :n] = k.table[0, :n]
        shares[k.table[0, :n]] += 1
    pool = np.concatenate([k.rng.permutation(k.n_pages).astype(np.int32), np.full(7, -9, np.int32)])
    return k, pool, (shares if shared else None)


def run_free(k, pool, shares, start, keep, **kw):
    free, sh = i32(pool), None if shares is None else i32(shares)
    info = rsa.page_free(i32(k.table), i32(k.lens), i32(keep), free, i64([start]), k.page, k.n_pages, shares=sh, **kw)
    return free.cpu().numpy(), None if sh is None else sh.cpu().numpy(), info.tolist()


@pytest.mark.parametrize("lens,keep,page,sharing", [
    ([40], [0], 16, None), ([40], [40], 16, None), ([40], [33], 16, None), ([40], [32], 16, None), ([40, 0, 100, 5], [17, 0, 0, 5], 16, None),
    ([100, 90, 80, 70], [0, 0, 80, 70], 16, {1: 3, 2: 2}),       # both users of a page, and one that is left
    ([100, 90, 80, 70], [0, 0, 0, 0], 16, {1: 3, 2: 2, 3: 4}), ([100, 90, 80, 70], [100, 0, 0, 33], 16, {1: 5, 2: 4, 3: 4}),
    ([1000] * 300, [0, 500] * 150, 16, {r: 30 for r in range(1, 200)}), ([5000] * 40, [0, 128] * 20, 16, None),
    ([3] * 5000, [0, 3, 1, 2, 0] * 1000, 128, None), ([60000, 70000], [1, 0], 16, {1: 3000}),
])
def test_free_matches_the_definition(lens, keep, page, sharing):
    need_cuda()
    k, pool, shares = free_case(lens, keep, page, sharing is not None, sharing=sharing)
    for start in (len(pool), len(pool) - 7):
        want = dr.free_pages(k.table, k.lens, keep, pool, start, shares, page, k.n_pages)
        got = run_free(k, pool, shares, start, keep)
        rsa.check_device_error()
        assert got[2] == want[2] and got[2][0] == 0
        assert np.array_equal(got[0], want[0])
        assert shares is None or np.array_equal(got[1], want[1])


@pytest.mark.parametrize("many", [False, True], ids=["one", "cluster"])
def test_pages_that_cannot_be_given_back_change_nothing(many):
    need_cuda()
    n = 400 if many else 4
    lens, keep = [100, 90, 80, 70] * (n // 4), [0, 10, 0, 0] * (n // 4)
    k, pool, shares = free_case(lens, keep, 16, True, sharing={1: 3, 2: 2})
    freed = dr.free_pages(k.table, k.lens, keep, pool, len(pool), shares, 16, k.n_pages)[2][1]
    for start, status in ((freed, 0), (freed - 1, 6), (0, 6), (-1, 6), (len(pool) + 1, 6), (-(1 << 62), 6), (1 << 62, 6)):
        got = run_free(k, pool, shares, start, keep)
        assert got[2] == ([0, freed, got[2][2], 0] if status == 0 else [6, 0, 0, start])
        if status:
            assert np.array_equal(got[0], pool) and np.array_equal(got[1], shares)
    for r, a, b in ((0, -1, 0), (1, 90, 91), (2, -5, -6), (3, 1 << 30, 0), (3, 70, -1)):
        k.lens[r], was, keep[r], kept_ = a, k.lens[r], b, keep[r]
        got = run_free(k, pool, shares, len(pool), keep)
        assert got[2] == [1, 0, 0, len(pool)]
        assert np.array_equal(got[0], pool) and np.array_equal(got[1], shares)
        k.lens[r], keep[r] = was, kept_
    rsa.check_device_error()


def test_free_reports_bad_pages_and_pages_given_back_too_often():
    need_cuda()
    for shared in (True, False):
        k, pool, shares = free_case([40, 40], [0, 0], 16, shared)
        k.table[0, 1] = 1 << 29
        got = run_free(k, pool, shares, 30, [0, 0])
        assert f"site code 0x9e, first bad index {1 << 29})" in reported()
        want = sorted([*k.table[0, [0, 2]], *k.table[1, :3]])
        assert got[2] == [0, 5, 6, 25] and got[0][25:30].tolist() == want
        k.table[0, 1] = twice = k.table[1, 1]
        got = run_free(k, pool, shares, 30, [0, 0])
        assert f"site code 0x9f, first bad index {twice})" in reported()
        assert got[2] == [0, 5, 6, 25] and got[0][25:30].tolist() == want
        assert not shared or (got[1] == 0).all()


def test_free_forms_and_refusals():
    need_cuda()
    k, pool, shares = free_case([40, 100], [0, 50], 16, False)
    want = dr.free_pages(k.table, k.lens, [0, 50], pool, 30, None, 16, k.n_pages)
    table = torch.full((2, 50), 3, dtype=torch.int32, device="cuda")
    table[:, 9:9 + k.table.shape[1]] = i32(k.table)
    free, info, side = i32(pool), i64([1, 2, 3, 4]), torch.cuda.Stream()
    args = [table[:, 9:9 + k.table.shape[1]], i32(k.lens), i32([0, 50]), free, i64([30]), 16, k.n_pages]
    torch.cuda.synchronize()
    got = rsa.page_free(*args, out=info, stream=side)
    side.synchronize()
    assert got is info and info.tolist() == want[2] and np.array_equal(free.cpu().numpy(), want[0])
    for at, bad in ((0, args[0].long()), (0, args[0][:1]), (1, args[1][:1]), (2, args[1].long()), (3, free.long()), (4, None), (4, i32([1])),
                    (4, i64([])), (5, 17), (6, 0), (6, (1 << 23) + 1), (3, args[1])):
        a = list(args)
        a[at] = bad
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.page_free(*a)
    for kw in (dict(shares=i32([0])), dict(out=i64([1])), dict(shares=free[:k.n_pages])):
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.page_free(*args, **kw)
    rsa.check_device_error()


def test_free_of_many_pages_in_the_bitmap():
    # the largest pool: 2^23 pages, ids at both ends and at the parts' borders
    need_cuda()
    n = 1 << 23
    ids = [0, 31, 32, n // 8 - 1, n // 8, n // 2, n - 1, 5 * (n // 8), 5 * (n // 8) - 1]
    table, free = i32([ids]), torch.full((50,), -4, dtype=torch.int32, device="cuda")
    for shares in (None, torch.zeros(n, dtype=torch.int32, device="cuda")):
        info = rsa.page_free(table, i32([len(ids) * 16]), i32([0]), free, i64([50]), 16, n, shares=shares)
        assert info.tolist() == [0, len(ids), len(ids), 50 - len(ids)] and free[50 - len(ids):].tolist() == sorted(ids)
    rsa.check_device_error()


def test_offsets_beyond_32_bits():
    # caches of 2^31 elements and more: forked and compacted at their far end
    need_cuda()
    page, Hkv, d, layers = 128, 2, 128, 3
    n_pages = (1 << 30) // (page * Hkv * d) + 40
    kc, vc = (torch.zeros(layers, n_pages, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b, c = n_pages - 3, n_pages - 2, n_pages - 1
    for x in (kc, vc):
        x[:, a:] = torch.randn(layers, 3, Hkv, page, d, generator=g, device="cuda").to(BF)
    was = [x[:, a:].clone() for x in (kc, vc)]
    table, kv = i32([[a, b], [0, 0]]), i32([page + 9, 0])
    info = rsa.page_fork(kc, vc, table, kv, i32([0]), i32([1]), i32([c]), shares=torch.zeros(n_pages, dtype=torch.int32, device="cuda"))
    assert info.tolist() == [0, 1, 1, 1] and table.tolist() == [[a, b], [a, c]]
    for x, w in zip((kc, vc), was):
        assert torch.equal(x[:, c, :, :9], w[:, 1, :, :9]) and torch.equal(x[:, c, :, 9:], w[:, 2, :, 9:]) and torch.equal(x[:, a:c], w[:, :2])
    got = rsa.cache_compact(kc, vc, table, i32([page - 1, 0]), kv, i32([[3, 9], [0, 0]]), i32([2, 0]))
    assert got.tolist() == [page + 1, 0]
    for x, w in zip((kc, vc), was):
        assert torch.equal(x[:, a, :, page - 1], w[:, 1, :, 2]) and torch.equal(x[:, b, :, 0], w[:, 1, :, 8])
        assert torch.equal(x[:, b, :, 1:], w[:, 1, :, 1:]) and not x[:, :10].any()
    rsa.check_device_error()
