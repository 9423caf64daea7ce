"""Steps after a window of the cached tokens was kept, whose keys keep their rotation: decode steps and a drafted
one, their positions moved on by what each request has dropped."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731


def on(positions, cu_new, dropped):
    """The positions of requests that have dropped tokens."""
    row = torch.arange(positions.numel(), dtype=torch.int32, device="cuda")
    return positions + dropped[torch.searchsorted(cu_new[1:], row, right=True).clamp_(max=dropped.numel() - 1)]


@pytest.mark.parametrize("dtype,d,page", [(BF, 128, 16), (F, 64, 32)])
def test_steps_after_a_window(dtype, d, page):
    need_cuda()
    g = torch.Generator().manual_seed(d)
    R, Hq, Hkv, n_pages, max_pages, pos0 = 3, 4, 2, 40, 8, 5
    table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")
    free, start = torch.randperm(n_pages, generator=g).int().cuda(), i64([0])
    kc, vc = (torch.full((1, n_pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    cs = rsa.rope_table(400, d)
    cached, dropped = i32([0] * R), i32([0] * R)
    held = [[] for _ in range(R)]  # (position, raw key, value) of every kept token

    def step(new, parent=None):
        """A step of `new` tokens a request: what the cache then holds is compared with keys rotated by the tokens'
        own positions, and the attention with its definition."""
        nonlocal start
        T = sum(new)
        q, k, v = (torch.randn(T, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
        plan = rsa.page_plan(cached, i32(new), table, free, page, n_pages, T, free_start=start, pos0=pos0)
        tree = rsa.tree_plan(i32(parent), plan.cu_new, plan.kv_len, 8, pos0=pos0) if parent else None
        pos = on((tree or plan).positions, plan.cu_new, dropped)
        ko = torch.empty_like(k)
        qo, _ = rsa.qk_norm_rope(q, k, None, None, pos, cs, v=v, slot_map=plan.slot_map, k_cache=kc[0], v_cache=vc[0], k_out=ko)
        args = (qo, kc[0], vc[0], plan.cu_new, table, plan.kv_len)
        out, lse = rsa.tree_attn(*args, tree.mask) if parent else rsa.prefix_attn(*args)
        rsa.check_device_error()
        cu = plan.cu_new.tolist()
        lens = plan.kv_len.tolist()
        at = [0] * T
        for r in range(R):
            follow = max([p for p, _, _ in held[r]], default=pos0 - 1) + 1  # behind all that is kept
            for i in range(cu[r], cu[r + 1]):
                back = parent[i] if parent else i - cu[r] - 1
                at[i] = follow if back < 0 else at[cu[r] + back] + 1
        assert pos.tolist() == at
        for x, y in ((q, qo), (k, ko)):
            want, bound = ref.norm_rope(ref.to64(x), None, np.array(at), ref.to64(cs), 1e-6)
            assert (np.abs(ref.to64(y) - want) <= bound + ref.half_step(dtype) * (np.abs(want) + bound)).all()
        rows = [[*((a, b) for _, a, b in held[r]), *zip(ref.to64(ko)[cu[r]:cu[r + 1]], ref.to64(v)[cu[r]:cu[r + 1]])] for r in range(R)]
        dense = [np.stack([x[c] for y in rows for x in y])[:, :, None] for c in (0, 1)]
        first = np.concatenate([[0], np.cumsum(lens)])
        dense_table = np.array([[first[r] + min(j, lens[r] - 1) for j in range(max(lens))] for r in range(R)])
        if parent:
            want = dr.tree_attn(ref.to64(qo), *dense, cu, dense_table, lens, tree.mask.cpu().numpy(), np.arange(0), 0)
        else:
            want = ref.prefix_attn(ref.to64(qo), *dense, cu, dense_table, lens, np.arange(0), 0)
        ref.assert_prefix_attn(out, lse, want, dtype)
        for r in range(R):
            held[r] += [(at[i], ref.to64(ko)[i], ref.to64(v)[i]) for i in range(cu[r], cu[r + 1])]
        start = plan.info[3:]
        return plan.kv_len

    def keep(base, lens, lists):
        """Own token base[r] + keep of each request's list stays; the others go, and their pages."""
        nonlocal start, cached
        m = max(1, *(len(x) for x in lists))
        new_len = rsa.cache_compact(kc, vc, table, i32(base), lens, i32([x + [0] * (m - len(x)) for x in lists]), i32([len(x) for x in lists]))
        info = rsa.page_free(table, lens, new_len, free, start, page, n_pages)
        rsa.check_device_error()
        assert info[0] == 0 and new_len.tolist() == [b + len(x) for b, x in zip(base, lists)]
        for r in range(R):
            held[r][:] = held[r][:base[r]] + [held[r][base[r] + j] for j in lists[r]]
        start = info[3:]
        cached = new_len

    cached = step([70, 50, 9])
    for r in range(2):  # twice, so that what is dropped adds up
        lens = cached.tolist()
        before = cached
        keep([0] * R, before, [[0, 1, 2, 3, *range(lens[0] - 21, lens[0])], list(range(lens[1] - 30, lens[1])), list(range(lens[2]))])
        dropped += before - cached
        cached = step([1, 7, 3])
        cached = step([2, 1, 1])
    assert min(dropped.tolist()[:2]) > 0 and dropped[2] == 0
    # a drafted step: dropped tokens of the tree do not count
    base = cached.tolist()
    lens = step([5, 4, 3], parent=[-1, 0, 0, 2, 1, -1, -1, 1, 2, -1, 0, 0])
    keep(base, lens, [[0, 2, 3], [1, 2], []])
    cached = step([1, 2, 3])
