"""page_free and page_fork from several host threads at once, with calls that want different
amounts of shared memory of the same kernel: neither may take the other's away."""
import threading

import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

CALLS = 2000


def arange(n):
    return torch.arange(n, dtype=torch.int32, device="cuda")


def full(n, v, dtype=torch.int32):
    return torch.full((n,), v, dtype=dtype, device="cuda")


def freeing(R, max_pages, n_pages):
    """A call that gives every request's second page back, and what it has to leave."""
    table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[:, 1] = arange(R), arange(R) + (n_pages - R)
    kv, keep, free, start = full(R, 32), full(R, 16), full(R + 5, -1), full(1, R + 2, torch.int64)
    want = torch.cat([full(2, -1), arange(R) + (n_pages - R), full(3, -1)])
    return (lambda: rsa.page_free(table, kv, keep, free, start, 16, n_pages)), [0, R, R, 2], lambda: torch.equal(free, want)


def forking(R, F):
    """F requests of one full page, each forked into a row of its own."""
    kc, vc = (torch.zeros(R, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, kv = arange(R)[:, None].contiguous(), full(R, 16)
    src, dst, free, shares = arange(F), arange(F) + F, full(1, 0), full(R, 0)
    want = torch.cat([arange(F), arange(F), arange(R)[2 * F:]])[:, None]
    return (lambda: rsa.page_fork(kc, vc, table, kv, src, dst, free, shares=shares)), [0, F, 0, 0], lambda: torch.equal(table, want)


@pytest.mark.parametrize("make,one,other", [
    (freeing, (2, 2, 700000), (3, 2, 400000)),              # short lists: the bitmap alone is large
    (freeing, (16000, 9, 200000), (5000, 27, 200000)),      # long lists
    (freeing, (2, 2, 1 << 23), (16000, 2, 790000)),         # more pages than one CTA's bitmap holds
    (forking, (16384, 8000), (5000, 2400)),
], ids=["free, short lists", "free, long lists", "free, many pages", "fork"])
def test_threads_with_different_amounts_of_shared_memory(make, one, other):
    need_cuda()
    work = [make(*one), make(*other), make(*one), make(*other)]
    torch.cuda.synchronize()
    ready, errors, info = threading.Barrier(4), [], [None] * 4

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ready.wait()
                for _ in range(CALLS):
                    info[i] = work[i][0]()
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, want, as_it_should_be), got in zip(work, info):
        assert got.tolist() == want and as_it_should_be()
    rsa.check_device_error()
