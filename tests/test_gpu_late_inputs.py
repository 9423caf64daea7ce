"""The calls for drafted tokens and the keeping of pages on inputs that another stream writes late: their launches
may begin early on their own stream, but not before an event that the stream waits for."""
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def calls():
    """name -> (inputs that are written late, a call on them and on copies of what it changes)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    kc, vc = (torch.randn(2, 40, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(14, 4, 64, generator=g, device="cuda").bfloat16()
    table, kv, cu = torch.randperm(40, generator=g, device="cuda").int()[:30].view(3, 10).contiguous(), i32([100, 60, 37]), i32([0, 6, 10, 14])
    parent = i32([-1, 0, 0, 1, 2, 4, -1, -1, 0, 1, -1, 0, 1, 2])
    mask = rsa.tree_plan(parent, cu, kv, 8).mask
    cached, keep, keep_len = i32([94, 56, 33]), i32([[0, 2, 4], [1, 3, 0], [2, 0, 0]]), i32([3, 2, 1])
    pool, start, shares, dst = torch.arange(40, dtype=torch.int32, device="cuda"), torch.tensor([30], device="cuda"), i32([0] * 40), i32([2])

    def compact(base, n):
        k, v = kc.clone(), vc.clone()
        return rsa.cache_compact(k, v, table, base, kv, keep, n), k, v

    def free(lens, kept):
        p = pool.clone()
        return rsa.page_free(table, lens, kept, p, start, 16, 40), p

    def fork(lens, src):
        k, v, t, n, s = kc.clone(), vc.clone(), table.clone(), lens.clone(), shares.clone()
        return rsa.page_fork(k, v, t, n, src, dst, pool, free_start=start, shares=s), k, v, t, n, s
    return {"tree_plan": ((parent, cu, kv), lambda *a: rsa.tree_plan(*a, 8)),
            "tree_attn": ((q, cu, kv, mask), lambda a, b, c, m: rsa.tree_attn(a, kc[0], vc[0], b, table, c, m)),
            "cache_compact": ((cached, keep_len), compact), "page_free": ((kv, i32([90, 0, 20])), free), "page_fork": ((kv, i32([1])), fork)}


@pytest.mark.parametrize("name", ["tree_plan", "tree_attn", "cache_compact", "page_free", "page_fork"])
def test_inputs_that_another_stream_writes_late(name):
    need_cuda()
    args, call = calls()[name]
    want = call(*args)
    late = [torch.zeros_like(a) for a in args]
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    call(*late)  # (loaded before the race)
    torch.cuda.synchronize()
    for stream in (mine, torch.cuda.default_stream()):
        for x in late:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # some 10 ms
            for x, a in zip(late, args):
                x.copy_(a)
            ready = side.record_event()
        with torch.cuda.stream(stream):
            torch.zeros(1, device="cuda").add_(1)  # a kernel of its own just before
            stream.wait_event(ready)
            got = call(*late)
        torch.cuda.synchronize()
        rsa.check_device_error()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("name", ["tree_plan", "tree_attn", "cache_compact", "page_free", "page_fork"])
def test_captured_inputs_that_another_stream_writes_late(name):
    need_cuda()
    args, call = calls()[name]
    want = call(*args)
    late = [torch.zeros_like(a) for a in args]
    call(*late)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in late:
            x.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)
            for x, a in zip(late, args):
                x.copy_(a)
        torch.zeros(1, device="cuda").add_(1)
        torch.cuda.current_stream().wait_stream(side)
        got = call(*late)
        again = call(*late)
    for _ in range(3):
        for x in (*got, *again):
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(got, again, want):
            assert torch.equal(x, z) and torch.equal(y, z)
    rsa.check_device_error()
