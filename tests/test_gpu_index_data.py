"""What index data outside its range leaves behind: the first offender's site and
value in rsa_check_device_error's text, and every other row as it would have been."""
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
from test_gpu_prefix_attn import Batch

pytestmark = pytest.mark.gpu

INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731


def reported():
    with pytest.raises(rsa.RsaError) as e:
        rsa.check_device_error()
    rsa.check_device_error()  # read and cleared
    assert e.value.status == 3
    return str(e.value)


def rotate(position, **kw):
    x = torch.randn(3, 2, 64, device="cuda")
    rsa.qk_norm_rope(x, x, None, None, i64([0, position, 1]), rsa.rope_table(8, 64), **kw)


def write(slot):
    v = torch.randn(3, 2, 64, device="cuda")
    caches = [torch.zeros(2, 2, 16, 64, device="cuda") for _ in range(2)]
    rotate(2, v=v, slot_map=i64([0, slot, 1]), k_cache=caches[0], v_cache=caches[1])


def attend(dtype=torch.float32, page=1, length=40, cu=1, first=0):
    q = torch.randn(1, 4, 64, device="cuda").to(dtype)
    kc, vc = (torch.randn(6, 2, 16, 64, device="cuda").to(dtype) for _ in range(2))
    rsa.prefix_attn(q, kc, vc, i32([first, cu]), i32([[0, page, 2]]), i32([length]))


def plan(page):
    rsa.page_plan(i32([0]), i32([1]), i32([[-1]]), i32([page]), 16, 6, 1)


@pytest.mark.parametrize("fault,site", [
    (lambda x: plan(x), 0x90), (lambda x: rotate(x), 0x91), (lambda x: attend(length=x), 0x94), (lambda x: attend(page=x), 0x95),
    (lambda x: attend(torch.bfloat16, page=x), 0x95),
], ids=["plan", "position", "kv_len", "page", "page_bf"])
@pytest.mark.parametrize("value", [-1, 99999, -77])
def test_site_and_value_are_the_offenders(fault, site, value):
    need_cuda()
    rsa.check_device_error()
    fault(value)
    assert f"site code 0x{site:02x}, first bad index {value})" in reported()


def test_slots_and_query_rows():
    need_cuda()
    write(5000)
    assert "site code 0x92, first bad index 5000)" in reported()
    attend(cu=-1)
    assert "site code 0x93, first bad index -1)" in reported()
    attend(cu=7)
    assert "site code 0x93, first bad index 7)" in reported()
    attend(first=-4)    # the bad one of the two
    assert "site code 0x93, first bad index -4)" in reported()


def test_the_first_of_two_is_kept():
    need_cuda()
    rotate(-1)          # (a -1 is a value like any other)
    rotate(77)
    assert "site code 0x91, first bad index -1)" in reported()
    rotate(99)
    write(5000)
    assert "site code 0x91, first bad index 99)" in reported()
    write(5000)
    rotate(-1)
    assert "site code 0x92, first bad index 5000)" in reported()
    attend(cu=-1)       # 0x93 and, as the lengths no longer fit, perhaps others
    attend(length=-5)
    assert "site code 0x93, first bad index -1)" in reported()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf", "f"])
@pytest.mark.parametrize("where", [1, 9], ids=["full tile", "short tile"])
@pytest.mark.parametrize("page", [INT_MIN, INT_MIN + 1, -1, INT_MAX])
def test_any_page_id_out_of_range_is_reported(dtype, where, page):
    # 150 keys in pages of 16: a tile of 128, and a shorter one of 22
    need_cuda()
    b = Batch([1, 1, 1], [40, 150, 60], 30, 4, 2, 64, 16, dtype)
    want, wl = b.check()
    b.table[1, where] = page
    out, lse = b.run()
    assert f"site code 0x95, first bad index {page})" in reported()
    keep = [0, 2]
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf", "f"])
def test_rows_that_do_not_ascend_leave_the_others_right(dtype):
    # request 1 is forced to the batch's end, where request 2 then has no rows: request 0 is as it was
    need_cuda()
    b = Batch([1, 1, 1], [40, 50, 60], 30, 4, 2, 64, 16, dtype)
    want, wl = b.check()
    b.cu = torch.tensor([0, 1, 1 << 30, 3], dtype=torch.int32)
    out, lse = b.run()
    assert "site code 0x93, first bad index" in reported()
    assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0])
