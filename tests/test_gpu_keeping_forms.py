"""page_fork and page_free where the tests of their definitions do not go: long lists of forks
with several faults at once, lists with entries that are no fork."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
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
