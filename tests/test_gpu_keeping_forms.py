"""page_fork and page_free where the tests of their definitions do not go: long lists of forks
with several faults at once."""
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
