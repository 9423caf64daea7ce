"""Requests that share pages, of which one keeps a window and one is cut back and grows again: by way of a fork into
a free row, without a trace in the others' rows."""
import numpy as np
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.mark.parametrize("dtype,page", [(BF, 16), (F, 64)])
def test_requests_that_share_pages_are_compacted_and_grow_again_beside_the_others(dtype, page):
    need_cuda()
    Hkv, d, layers, n_pages, R = 2, 64, 2, 60, 5
    g = torch.Generator().manual_seed(page)
    kc, vc = (torch.randn(layers, n_pages, Hkv, page, d, generator=g).to(dtype).cuda() for _ in range(2))
    table = torch.full((R, 8), -1, dtype=torch.int32, device="cuda")
    free, shares = torch.randperm(n_pages, generator=g).int().cuda(), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    n = 4 * page + 5
    plan = rsa.page_plan(i32([0] * R), i32([n, 0, 0, 0, 0]), table, free, page, n_pages, n)
    kv, start = plan.kv_len, plan.info[3:]

    def rows(r):
        """[tokens, layers, Hkv, d], keys and values."""
        at = torch.arange(int(kv[r]), device="cuda")
        return [c[:, table[r, at // page].long(), :, at % page].clone() for c in (kc, vc)]

    def ends(*gone):
        """These requests end."""
        nonlocal start
        left = kv.clone()
        left[list(gone)] = 0
        info = rsa.page_free(table, kv, left, free, start, page, n_pages, shares=shares)
        assert info[0] == 0
        start = info[3:]
        kv.copy_(left)

    def fork(a, b, counted):
        nonlocal start
        info = rsa.page_fork(kc, vc, table, kv, i32([a]), i32([b]), free, free_start=start, shares=shares if counted else None)
        assert info[0] == 0
        start = info[3:]

    fork(0, 1, True)
    fork(0, 2, True)
    was = rows(0)
    # request 1 keeps a window: its pages become its own first
    fork(1, 3, False)
    ends(1)
    kept = [1, 2, *range(2 * page, n)]
    cut = rsa.cache_compact(kc, vc, table, i32([0] * R), kv, i32([kept] * R), i32([0, 0, 0, len(kept), 0]))
    cut = torch.where(i32([0, 0, 0, 1, 0]) > 0, cut, kv)
    info = rsa.page_free(table, kv, cut, free, start, page, n_pages, shares=shares)
    assert info[0] == 0
    start = info[3:]
    kv.copy_(cut)
    for x, y, z, w in zip(rows(0), rows(2), rows(3), was):
        assert torch.equal(x, w) and torch.equal(y, w) and torch.equal(z, w[kept])
    # request 2 is cut back into a shared page and grows again: a page of its own takes the partial one's place
    cut = kv.clone()
    cut[2] = 2 * page + 3
    info = rsa.page_free(table, kv, cut, free, start, page, n_pages, shares=shares)
    start = info[3:]
    kv.copy_(cut)
    fork(2, 4, True)
    ends(2)
    new = torch.randn(2, 20, Hkv, d, generator=g).to(dtype).cuda()
    plan = rsa.page_plan(kv, i32([0, 0, 0, 0, 20]), table, free, page, n_pages, 20, free_start=start)
    start = plan.info[3:]
    for c, x in zip((kc, vc), new):
        c[:, plan.slot_map // page, :, plan.slot_map % page] = x[:, None]
    kv = plan.kv_len
    for x, z, y, w, fresh in zip(rows(0), rows(3), rows(4), was, new):
        assert torch.equal(x, w) and torch.equal(z, w[kept])
        m = 2 * page + 3
        assert torch.equal(y[:m], w[:m]) and all(torch.equal(y[m:, i], fresh) for i in range(layers))
    users = np.zeros(n_pages, int)
    for r in range(R):
        np.add.at(users, table[r, :-(-int(kv[r]) // page)].cpu().numpy(), 1)
    assert np.array_equal(np.maximum(users - 1, 0), shares.cpu().numpy())
    ends(0, 3, 4)
    assert not shares.any() and int(start) == 0 and sorted(free.tolist()) == list(range(n_pages))
    rsa.check_device_error()
