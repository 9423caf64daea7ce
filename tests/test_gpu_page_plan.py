"""page_plan on the GPU against the plain loop: every number equal."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu


def run(cached, new, page, max_pages, free, max_tokens, start=None, pos0=0, n_pages=None, table=None, stride=None):
    R = len(cached)
    if table is None:
        # old pages: distinct ids above the free ones
        table = np.full((R, max_pages), -1, np.int32)
        nxt = 10000
        for r in range(R):
            for j in range(min(max_pages, -(-max(cached[r], 0) // page))):
                table[r, j] = nxt
                nxt += 1
    n_pages = 1 << 20 if n_pages is None else n_pages
    wide = np.full((R, stride or max_pages), -7, np.int32)
    wide[:, :max_pages] = table
    dev = torch.from_numpy(wide).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    p = rsa.page_plan(i32(cached), i32(new), dev[:, :max_pages], i32(free), page, n_pages, max_tokens,
                      free_start=None if start is None else torch.tensor([start], device="cuda"), pos0=pos0)
    want = ref.page_plan(cached, new, table, free, page, max_tokens, start or 0, pos0)
    torch.cuda.synchronize()
    got = (dev[:, :max_pages], *p)
    for name, g, w in zip(("table", "cu_new", "kv_len", "slot_map", "positions", "info"), got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    if stride:
        assert (dev[:, max_pages:] == -7).all()  # beside the rows nothing is written
    return p


@pytest.mark.parametrize("R,page,new,old,pad,seed", [
    (1, 16, 1, 0, 0, 0), (1, 64, 1, 63, 3, 1), (1, 64, 1, 64, 0, 2), (3, 128, 300, 1000, 5, 3), (8, 32, 1, 500, 1, 4),
    (33, 16, 40, 90, 0, 5), (513, 16, 5, 200, 7, 6), (1025, 64, 3, 70, 2, 7), (16384, 16, 2, 40, 1, 8), (2, 16, 70000, 10, 3, 9),
])
def test_matches_the_loop(R, page, new, old, pad, seed):
    need_cuda()
    rng = np.random.default_rng(seed)
    cached = [int(x) for x in rng.integers(0, old + 1, R)]
    n = [int(x) for x in rng.integers(0 if R > 2 else 1, new + 1, R)]  # some requests have no new token
    max_pages = max(-(-(c + k) // page) for c, k in zip(cached, n)) or 1
    need = sum(-(-(c + k) // page) - -(-c // page) for c, k in zip(cached, n))
    free = [int(x) for x in rng.permutation(need + 9)]
    run(cached, n, page, max_pages, free, max(1, sum(n) + pad), start=4, pos0=77, stride=max_pages + 3)
    rsa.check_device_error()


def test_edges_of_pages_and_requests_without_tokens():
    need_cuda()
    free = list(range(100, 140))
    run([0, 0, 16, 15, 17, 32], [0, 16, 0, 1, 15, 1], 16, 4, free, 40)
    run([0, 0, 0], [0, 0, 0], 16, 2, free, 5)                # a step without tokens
    run([5, 5], [0, 0], 16, 1, [], 1)                        # ... and without free pages
    run([16 * 4 - 1], [1], 16, 4, [], 1)                     # the last row of the last page
    rsa.check_device_error()


@pytest.mark.parametrize("why,kw", [
    ("negative cached length", dict(cached=[3, -1], new=[1, 1])),
    ("negative new length", dict(cached=[3, 4], new=[1, -5])),
    ("row of the table too short", dict(cached=[30, 1], new=[3, 1])),
    ("free pages do not suffice", dict(cached=[0, 0], new=[32, 17], free=[1, 2, 3])),
    ("start behind the free pages", dict(cached=[0, 0], new=[1, 1], start=9)),
    ("negative start", dict(cached=[0, 0], new=[1, 1], start=-1)),
    ("more tokens than rows", dict(cached=[0, 0], new=[5, 4])),
    ("lengths whose sum passes 32 bits", dict(cached=[0, 0], new=[2147483647, 2147483647])),
])
def test_a_step_that_cannot_be_planned_changes_nothing(why, kw):
    need_cuda()
    kw = dict(dict(free=[1, 2, 3, 4], start=0), **kw)
    p = run(kw["cached"], kw["new"], 16, 2, kw["free"], 8, start=kw["start"])
    assert p.info[0].item() != 0 and int(p.info[0]) in rsa.PLAN_STATUS
    rsa.check_device_error()


def test_bad_page_ids_leave_no_slot_and_are_reported():
    need_cuda()
    # request 0 goes on in page 999999 of its table, request 1 gets free page -3: neither is a page of the cache
    table = np.array([[999999, -1], [-1, -1], [7, -1]], np.int32)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    p = rsa.page_plan(i32([3, 0, 3]), i32([2, 1, 1]), torch.from_numpy(table).cuda(), i32([-3]), 16, 100, 5)
    with pytest.raises(rsa.RsaError) as e:
        rsa.check_device_error()
    assert e.value.status == 3 and "bounds check" in str(e.value)
    assert p.slot_map.tolist() == [-1, -1, -1, 7 * 16 + 3, -1] and p.info.tolist() == [0, 4, 1, 1]
    rsa.check_device_error()  # read and cleared


def test_a_chain_of_steps_needs_no_host():
    # kv_len and info feed the next step; two sets of outputs take turns, captured into one graph and replayed
    need_cuda()
    page, R, max_pages = 16, 5, 8
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(60, device="cuda").to(torch.int32)
    one = i32([1] * R)
    a = rsa.page_plan(i32([0, 3, 15, 16, 30]), i32([0] * R), table, free, page, 100, R,
                      free_start=torch.zeros(1, dtype=torch.int64, device="cuda"))
    # (lengths without pages: give the old tokens theirs first)
    old = rsa.page_plan(i32([0] * R), i32([0, 3, 15, 16, 30]), table, free, page, 100, 64, free_start=a.info[3:])
    new = lambda: rsa.PagePlan(torch.empty(R + 1, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda"),  # noqa: E731
                               *(torch.empty(n, dtype=torch.int64, device="cuda") for n in (R, R, 4)))
    x, y = new(), new()
    y.kv_len.copy_(old.kv_len)
    y.info.copy_(old.info)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        rsa.page_plan(y.kv_len, one, table, free, page, 100, R, free_start=y.info[3:], out=x)
        rsa.page_plan(x.kv_len, one, table, free, page, 100, R, free_start=x.info[3:], out=y)
    lens, t = [0, 3, 15, 16, 30], table.cpu().numpy().copy()
    start, fl = int(old.info[3]), free.tolist()
    for _ in range(6):
        g.replay()
        for _ in range(2):
            t, cu, kv, slots, pos, info = ref.page_plan(lens, [1] * R, t, fl, page, R, start)
            lens, start = kv.tolist(), int(info[3])
        torch.cuda.synchronize()
        np.testing.assert_array_equal(table.cpu().numpy(), t)
        assert y.kv_len.tolist() == lens and y.info.tolist() == info.tolist()
        assert y.slot_map.tolist() == slots.tolist() and y.positions.tolist() == pos.tolist()
    rsa.check_device_error()


def test_python_refuses_tensors_that_do_not_fit():
    need_cuda()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ok = (i32(3), i32(3), i32(3, 4), i32(9), 16, 50, 8)
    for at, bad in [(0, i32(3).long()), (1, i32(2)), (2, i32(2, 4)), (2, i32(4, 3).t()), (3, i32(3, 3)), (3, i32(18)[::2])]:
        args = list(ok)
        args[at] = bad
        with pytest.raises((ValueError, TypeError)):
            rsa.page_plan(*args)
    with pytest.raises(rsa.RsaError):
        rsa.page_plan(*ok[:4], 17, 50, 8)
    with pytest.raises(ValueError):
        rsa.page_plan(*ok, free_start=i32(1))
    with pytest.raises(ValueError):  # outputs made on the current stream for a bare handle of another
        rsa.page_plan(*ok, stream=torch.cuda.Stream().cuda_stream)
