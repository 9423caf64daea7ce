"""Drafted steps as a server runs them, captured and replayed: plan, tree plan, head norm
with cache write and tree attention in every layer, then the accepted tokens moved
together and the others' pages given back; requests fork and end between the steps.
The attention of every step is compared with its definition over the rows that the
accepted tokens had when they were written, and no page may get lost."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731


@pytest.mark.parametrize("dtype,d,page,prefix", [(torch.bfloat16, 128, 16, 40), (torch.bfloat16, 64, 64, 0), (torch.float32, 64, 16, 33)])
def test_captured_drafted_steps_with_forks(dtype, d, page, prefix):
    need_cuda()
    rng, g = np.random.default_rng(page + prefix), torch.Generator().manual_seed(d)
    R, Hq, Hkv, layers, tree, max_pages, n_pages, steps = 4, 4, 2, 2, 9, 12, 80, 10
    rows = R * tree + 3
    npre = -(-prefix // page)
    pool = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    prefix_pages, free = pool[:npre].clone(), pool[npre:].clone()
    kc, vc = (torch.full((layers, n_pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    for c in (kc, vc):
        for j in range(prefix):
            c[:, prefix_pages[j // page], :, j % page] = torch.randn(layers, Hkv, d, generator=g).to(dtype).cuda()
    table, shares = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    cs = rsa.rope_table(prefix + 400, d)
    x = [torch.zeros(rows, (Hq + 2 * Hkv) * d, dtype=dtype, device="cuda") for _ in range(layers)]
    qkv = lambda t: (t[:, :Hq * d].view(rows, Hq, d), t[:, Hq * d:-Hkv * d].view(rows, Hkv, d), t[:, -Hkv * d:].view(rows, Hkv, d))  # noqa: E731
    ko = [torch.zeros(rows, Hkv, d, dtype=dtype, device="cuda") for _ in range(layers)]
    cached, start = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    new, parent = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    keep, keep_len = torch.zeros(R, tree, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")

    def step():
        plan = rsa.page_plan(cached, new, table, free, page, n_pages, rows, free_start=start, pos0=prefix)
        t = rsa.tree_plan(parent, plan.cu_new, plan.kv_len, tree, pos0=prefix)
        res = []
        for n in range(layers):
            q, k, v = qkv(x[n])
            qo, _ = rsa.qk_norm_rope(q, k, None, None, t.positions, cs, v=v, slot_map=plan.slot_map, k_cache=kc[n], v_cache=vc[n], k_out=ko[n])
            res.append((qo, *rsa.tree_attn(qo, kc[n], vc[n], plan.cu_new, table, plan.kv_len, t.mask, prefix_pages=prefix_pages,
                                           prefix_len=prefix)))
        length = rsa.cache_compact(kc, vc, table, cached, plan.kv_len, keep, keep_len)
        info = rsa.page_free(table, plan.kv_len, length, free, plan.info[3:], page, n_pages, shares=shares)
        cached.copy_(length)
        start.copy_(info[3:])
        return plan, t, res, info

    # the kernels are loaded before the capture, by a step in which nothing is new
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, t, res, info = step()

    # every request's accepted rows of keys and values of each layer, in 64 bits
    pre = [[ref.to64(c[n])[prefix_pages.cpu().numpy()[np.arange(prefix) // page], :, np.arange(prefix) % page] for c in (kc, vc)]
           for n in range(layers)]
    held = [[[[], []] for _ in range(layers)] for _ in range(R)]

    def in_use():
        """Pages of the requests, each counted once, with what shares says of them."""
        t_, lens = table.cpu().numpy(), cached.tolist()
        users = np.zeros(n_pages, np.int64)
        for r in range(R):
            for p in t_[r, :-(-lens[r] // page)]:
                users[p] += 1
        assert np.array_equal(np.maximum(users - 1, 0), shares.cpu().numpy())
        return set(np.nonzero(users)[0].tolist())

    for i in range(steps):
        sizes = [int(rng.integers(1, tree + 1)) for _ in range(R)]
        if i == 3:
            sizes[2] = 0
        forests = [dr.random_forest(rng, n, 3) for n in sizes]
        paths = []
        for f in forests:  # a node's way from its root, or nothing accepted
            at, path = (int(rng.integers(0, len(f))) if f and rng.random() < 0.9 else -1), []
            while at >= 0:
                path.insert(0, at)
                at = f[at]
            paths.append(path)
        new.copy_(i32(sizes))
        flat = sum(forests, [])
        parent.fill_(77)
        parent[:len(flat)] = i32(flat)
        for r, p in enumerate(paths):
            keep[r, :len(p)] = i32(p)
        keep_len.copy_(i32([len(p) for p in paths]))
        for y in x:
            y.copy_(torch.randn(y.shape, generator=g).to(dtype))
        for _, out, _ in res:
            out.fill_(3)
        before = cached.tolist()
        graph.replay()
        torch.cuda.synchronize()
        rsa.check_device_error()
        assert plan.info[0] == 0 and info[0] == 0
        cu = np.concatenate([[0], np.cumsum(sizes)]).tolist()
        lens = [b + n for b, n in zip(before, sizes)]
        pos, mask = dr.tree_plan(flat, cu, lens, 1, rows, pos0=prefix)
        assert np.array_equal(t.positions.cpu().numpy(), pos) and np.array_equal(t.mask.cpu().numpy(), mask)
        for n in range(layers):
            qo, out, lse = res[n]
            k, v = ref.to64(ko[n]), ref.to64(qkv(x[n])[2])
            # a page of one row for each token: the prefix, then what each request holds and has drafted
            rows_of = [[*held[r][n][c], *(k, v)[c][cu[r]:cu[r + 1]]] for r in range(R) for c in (0, 1)]
            dense = [np.concatenate([pre[n][c], *(np.array(y).reshape(-1, Hkv, d) for y in rows_of[c::2])])[:, :, None] for c in (0, 1)]
            first = prefix + np.concatenate([[0], np.cumsum(lens)])
            dense_table = np.array([[first[r] + min(j, max(lens[r] - 1, 0)) for j in range(max(lens))] for r in range(R)])
            want = dr.tree_attn(ref.to64(qo), *dense, cu, dense_table, lens, mask, np.arange(prefix), prefix)
            ref.assert_prefix_attn(out, lse, want, dtype, cu[R])
            assert (out[cu[R]:] == 3).all()
            for r in range(R):
                for j in paths[r]:
                    held[r][n][0].append(k[cu[r] + j])
                    held[r][n][1].append(v[cu[r] + j])
        assert cached.tolist() == [b + len(p) for b, p in zip(before, paths)]
        used = in_use()
        left = free[int(start):].tolist()
        assert not used & set(left) and len(used) + len(left) == n_pages - npre and len(set(left)) == len(left)
        if i in (4, 7):
            # requests 1 and 3 end, and go on as copies of request 0
            end = cached.clone()
            end[1] = end[3] = 0
            freed = rsa.page_free(table, cached, end, free, start, page, n_pages, shares=shares)
            got = rsa.page_fork(kc, vc, table, cached, i32([0, 0]), i32([1, 3]), free, free_start=freed[3:], shares=shares)
            assert freed[0] == 0 and got[0] == 0
            start.copy_(got[3:])
            for r in (1, 3):
                held[r] = [[list(c) for c in y] for y in held[0]]
            in_use()
    # all requests end: every page is free again
    freed = rsa.page_free(table, cached, torch.zeros_like(cached), free, start, page, n_pages, shares=shares)
    assert freed[0] == 0 and freed[3] == 0 and sorted(free.tolist()) == sorted(pool[npre:].tolist()) and not shares.any()
    rsa.check_device_error()
