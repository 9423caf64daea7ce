"""page_fork and page_free where the tests of their definitions do not go: long lists of forks
with several faults at once, lists with entries that are no fork; pages given back wrongly in
each of the forms that the freeing takes, and more pages than it can list in shared memory."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
from test_gpu_index_data import reported
from test_gpu_page_keeping import Keeper, i32, i64

pytestmark = pytest.mark.gpu


# ---- page_fork -----------------------------------------------------------------------------

@pytest.mark.parametrize("F", [40, 250, 700])
@pytest.mark.parametrize("shared", [True, False], ids=["shared", "copied"])
def test_the_first_fault_that_applies_is_told_whichever_is_found_first(F, shared):
    # a bad length in one fork, a request both in src and in dst in another: always the latter, from all blocks' threads
    need_cuda()
    R = 2 * F + 1
    k = Keeper([20] * R, 16, layers=1, Hkv=1, extra=2 * F)
    sh = i32([0] * k.n_pages) if shared else None
    for long, both in ((0, F - 1), (F - 1, 0), (3, 33), (33, 3), (F // 2, F - 2)):
        src, dst, lens = list(range(F)), list(range(F, 2 * F)), list(k.lens)
        lens[long] = 1 << 30
        src[both] = F + (both + 1) % F
        want = dr.fork(k.plain(), k.table, lens, src, dst, k.free, k.start, None, 16)
        assert want[4] == [5, 0, 0, k.start]
        table, kv, free, start, src, dst = i32(k.table), i32(lens), i32(k.free), i64([k.start]), i32(src), i32(dst)
        infos = [rsa.page_fork(*k.dev, table, kv, src, dst, free, free_start=start, shares=sh) for _ in range(40)]
        assert torch.equal(torch.stack(infos), i64(want[4]).expand(40, 4)), (long, both)
        assert np.array_equal(table.cpu().numpy(), k.table) and kv.tolist() == lens and (sh is None or not sh.any())
        # the length alone
        src[both] = both
        info = rsa.page_fork(*k.dev, table, kv, src, dst, free, free_start=start, shares=sh)
        assert info.tolist() == [1, 0, 0, k.start]
    k.assert_caches(k.plain())
    rsa.check_device_error()


@pytest.mark.parametrize("shared", [True, False], ids=["shared", "copied"])
@pytest.mark.parametrize("F,forks", [(1, 0), (3, 1), (70, 0), (70, 33), (300, 7), (300, 290)])
def test_entries_that_are_no_fork(F, forks, shared):
    need_cuda()
    R, page = forks + 9, 16
    rng = np.random.default_rng(F + forks)
    lens = [int(rng.integers(0, 70)) for _ in range(9)] + [0] * forks
    R = max(R, F)  # (a call has no more entries than requests)
    lens += [0] * (R - len(lens))
    k = Keeper(lens, page, layers=2, Hkv=2, extra=forks * 5 + 3)
    src, dst = [int(rng.integers(0, 9)) for _ in range(forks)], [9 + f for f in rng.permutation(forks).tolist()]
    sh = np.zeros(k.n_pages, np.int32) if shared else None
    want = dr.fork(k.plain(), k.table, k.lens, src, dst, k.free, k.start, sh, page)
    at = sorted(rng.permutation(F)[:forks].tolist())  # the forks' order is kept
    s, d = [-1] * F, [-1] * F
    for i, f in enumerate(at):
        s[f], d[f] = src[i], dst[i]
    table, kv, sh = i32(k.table), i32(k.lens), i32(sh) if shared else None
    info = rsa.page_fork(*k.dev, table, kv, i32(s), i32(d), i32(k.free), free_start=i64([k.start]), shares=sh)
    rsa.check_device_error()
    assert info.tolist() == want[4] and want[4][0] == 0
    assert np.array_equal(table.cpu().numpy(), want[1]) and kv.tolist() == want[2]
    assert not shared or np.array_equal(sh.cpu().numpy(), want[3])
    k.assert_caches(want[0])
    # -1 in one of them alone is a request outside the batch
    for one in (s, d):
        was = one[0]
        (d if one is s else s)[0], one[0] = 0, -1
        assert rsa.page_fork(*k.dev, table, kv, i32(s), i32(d), i32(k.free), free_start=i64([k.start]), shares=sh)[0] == 5
        one[0] = was
        s[0] = d[0] = -1


def test_a_captured_call_forks_as_many_as_there_are():
    need_cuda()
    F, page, R = 6, 16, 10
    k = Keeper([40, 33, 7, 64] + [0] * 6, page, extra=40)
    table, kv, free, sh = i32(k.table), i32(k.lens), i32(k.free), i32([0] * k.n_pages)
    src, dst, start = i32([-1] * F), i32([-1] * F), i64([k.start])
    assert rsa.page_fork(*k.dev, table, kv, src, dst, free, free_start=start, shares=sh).tolist() == [0, 0, 0, k.start]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        info = rsa.page_fork(*k.dev, table, kv, src, dst, free, free_start=start, shares=sh)
        start.copy_(info[3:])
    state = [k.plain(), k.table, k.lens, None, [0, 0, 0, k.start]]
    shares = np.zeros(k.n_pages, np.int32)
    for forks in ([], [(0, 4)], [(1, 5), (3, 6), (1, 7)], [], [(4, 8), (2, 9)]):
        s, d = [a for a, _ in forks], [b for _, b in forks]
        src.copy_(i32(s + [-1] * (F - len(s))))
        dst.copy_(i32(d + [-1] * (F - len(d))))
        graph.replay()
        state = dr.fork(state[0], state[1], state[2], s, d, k.free, state[4][3], shares, page)
        shares = state[3]
        assert info.tolist() == state[4] and state[4][0] == 0
        assert np.array_equal(table.cpu().numpy(), state[1]) and kv.tolist() == state[2] and sh.tolist() == shares.tolist()
        k.assert_caches(state[0])
    rsa.check_device_error()


# ---- page_free -----------------------------------------------------------------------------

# few table entries; many of them, nearly all unused; more pages than a bitmap in one SM holds
FORMS = {"short": (500, 0), "long": (500, 140000), "many pages": (900001, 0)}


class Pool:
    """A table of pages all over the pool, whose rows may share their first pages with row 0 (`sharing`)."""

    def __init__(self, form, lens, sharing=None, page=16, seed=0):
        rng = np.random.default_rng(seed)
        self.n_pages, entries = FORMS[form]
        self.page, self.lens = page, list(lens)
        counts = [-(-n // page) for n in lens]
        ids = np.concatenate([[0, self.n_pages - 1, 31, 32], 40 + rng.permutation(self.n_pages - 50)[:sum(counts)]])[:sum(counts)]
        ids = rng.permutation(ids).astype(np.int32)
        self.table = np.full((len(lens), max(max(counts) + 1, -(-entries // len(lens)))), -(1 << 30), np.int32)
        at = 0
        for r, n in enumerate(counts):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.shares = np.zeros(self.n_pages, np.int32)
        for r, n in (sharing or {}).items():
            self.table[r, :n] = self.table[0, :n]
            self.shares[self.table[0, :n]] += 1
        self.pool = rng.integers(0, 1 << 20, sum(counts) + 9).astype(np.int32)

    def want(self, keep, start, shared):
        return dr.free_pages(self.table, self.lens, keep, self.pool, start, self.shares if shared else None, self.page, self.n_pages)

    def got(self, keep, start, shared):
        free, sh = i32(self.pool), i32(self.shares) if shared else None
        info = rsa.page_free(i32(self.table), i32(self.lens), i32(keep), free, i64([start]), self.page, self.n_pages, shares=sh)
        return free.cpu().numpy(), sh.cpu().numpy() if shared else None, info.tolist()


def assert_same(got, want):
    assert got[2] == want[2] and np.array_equal(got[0], want[0])
    assert want[1] is None or np.array_equal(got[1], want[1])


LENS, KEEP = [100, 90, 80, 70, 200, 0, 5] * 8, [100, 0, 10, 0, 33, 0, 0] * 8


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("shared", [True, False], ids=["counted", "plain"])
def test_freeing_with_and_without_room_in_each_form(form, shared):
    need_cuda()
    k = Pool(form, LENS, {8: 5, 15: 3, 22: 5, 43: 2} if shared else None)
    n = k.want(KEEP, len(k.pool), shared)[2][1]
    assert n > 50
    for start in (n, len(k.pool), n - 1, 0, -5, len(k.pool) + 1):
        want = k.want(KEEP, start, shared)
        assert want[2][0] == (0 if n <= start <= len(k.pool) else 6)
        assert_same(k.got(KEEP, start, shared), want)
    keep = list(KEEP)
    for r, length, kept in ((0, 100, 101), (55, -1, 0), (30, 16 * k.table.shape[1] + 1, 0), (17, 70, -2)):
        was, k.lens[r], keep[r] = (k.lens[r], keep[r]), length, kept
        want = k.want(keep, len(k.pool), shared)
        assert want[2] == [1, 0, 0, len(k.pool)]
        assert_same(k.got(keep, len(k.pool), shared), want)
        k.lens[r], keep[r] = was
    rsa.check_device_error()


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("shared", [True, False], ids=["counted", "plain"])
def test_bad_pages_and_pages_given_back_twice_in_each_form(form, shared):
    need_cuda()
    lens, keep = [40, 40, 64, 160], [0, 0, 16, 0]
    for bad in (-1, FORMS[form][0], 1 << 30, -(1 << 31)):
        k = Pool(form, lens)
        k.table[1, 1] = bad
        got = k.got(keep, len(k.pool), shared)
        assert f"site code 0x9e, first bad index {bad})" in reported()
        left = sorted([*k.table[0, :3], *k.table[1, [0, 2]], *k.table[2, 1:4], *k.table[3, :10]])
        start = len(k.pool) - len(left)
        assert got[2] == [0, len(left), len(left) + 1, start] and got[0][start:].tolist() == left and np.array_equal(got[0][:start], k.pool[:start])
    for twice in ([(0, 0, 1, 0)], [(3, 9, 3, 0)], [(0, 0, 1, 0), (0, 0, 2, 1), (0, 0, 3, 3), (0, 1, 3, 4), (2, 3, 3, 5)]):
        k = Pool(form, lens)
        for a, i, b, j in twice:
            k.table[b, j] = k.table[a, i]
        left = sorted({*k.table[0, :3].tolist(), *k.table[1, :3].tolist(), *k.table[2, 1:4].tolist(), *k.table[3, :10].tolist()})
        got = k.got(keep, len(k.pool), shared)
        text = reported()
        assert any(f"site code 0x9f, first bad index {k.table[a, i]})" in text for a, i, _, _ in twice)
        start = len(k.pool) - len(left)
        assert got[2] == [0, len(left), 19, start] and got[0][start:].tolist() == left and np.array_equal(got[0][:start], k.pool[:start])
        assert not shared or not got[1].any()
        # without room for them nothing is changed
        assert_same(k.got(keep, len(left) - 1, shared), (k.pool, k.shares if shared else None, [6, 0, 0, len(left) - 1]))
        assert not shared or "site code 0x9f" in reported()
    rsa.check_device_error()


@pytest.mark.parametrize("R,pages", [(1, 120000), (4, 100000)], ids=["short", "long"])
@pytest.mark.parametrize("shared", [True, False], ids=["counted", "plain"])
def test_more_pages_than_are_listed_in_shared_memory(R, pages, shared):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(R)
    n_pages = R * pages + 77
    table = torch.randperm(n_pages, generator=g, device="cuda")[:R * pages].int().view(R, pages).contiguous()
    free, shares = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    kv, keep = i32([pages * 16 - r for r in range(R)]), i32([16 * r for r in range(R)])
    info = rsa.page_free(table, kv, keep, free, i64([n_pages - 7]), 16, n_pages, shares=shares if shared else None)
    rsa.check_device_error()
    gone = torch.cat([table[r, r:] for r in range(R)]).sort().values
    start = n_pages - 7 - gone.numel()
    assert info.tolist() == [0, gone.numel(), gone.numel(), start]
    assert torch.equal(free[start:n_pages - 7], gone) and (free[:start] == -1).all() and (free[n_pages - 7:] == -1).all() and not shares.any()
