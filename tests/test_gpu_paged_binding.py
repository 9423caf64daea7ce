"""The compiled binding of the paged calls: outputs that the caller passes, streams
by their bare handles, and where the tensors that a call makes come from."""
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def step_of(d=64):
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, gq, gk = rand(7, 4, d), rand(7, 2, d), rand(7, 4, d), rand(7, 2, d)
    return (gq, gk, q, k, 1 + 0.1 * rand(d), 1 + 0.1 * rand(d), torch.arange(7, device="cuda"), rsa.rope_table(10, d))


def test_gradient_on_a_bare_handle_with_every_output_passed():
    # a handle says nothing about who holds its stream: only calls that make no tensors take one
    need_cuda()
    args = step_of()
    want = rsa.qk_norm_rope_bwd(*args)
    side = torch.cuda.Stream()
    out = dict(dq=torch.empty_like(args[2]), dk=torch.empty_like(args[3]), dq_weight=torch.empty(64, device="cuda"),
               dk_weight=torch.empty(64, device="cuda"), workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    got = rsa.qk_norm_rope_bwd(*args, **out, stream=side.cuda_stream)
    side.synchronize()
    for x, y, n in zip(got, want, ("dq", "dk", "dq_weight", "dk_weight")):
        assert x is out[n] and torch.equal(x, y)
    for n in out:
        with pytest.raises(ValueError):
            rsa.qk_norm_rope_bwd(*args, **{**out, n: None}, stream=side.cuda_stream)
    rsa.check_device_error()


def test_weight_gradients_that_the_caller_passes():
    need_cuda()
    args = step_of()
    want = rsa.qk_norm_rope_bwd(*args)
    dw = torch.full((64,), 9.0, device="cuda")
    got = rsa.qk_norm_rope_bwd(*args, dk_weight=dw)
    assert got[3] is dw and all(torch.equal(x, y) for x, y in zip(got, want))
    # a gradient of weights of ones, where they are not given
    ones = torch.ones(64, device="cuda")
    got = rsa.qk_norm_rope_bwd(*args[:4], None, None, *args[6:], dq_weight=dw)
    want = rsa.qk_norm_rope_bwd(*args[:4], ones, ones, *args[6:])
    assert got[2] is dw and got[3] is None and torch.equal(dw, want[2])
    for bad, err in ((torch.empty(32, device="cuda"), ValueError), (torch.empty(64, device="cuda").bfloat16(), ValueError),
                     (torch.empty(128, device="cuda")[::2], ValueError), (torch.empty(64), TypeError)):
        with pytest.raises(err):
            rsa.qk_norm_rope_bwd(*args, dq_weight=bad)
    rsa.check_device_error()


def test_tensors_that_a_call_makes_are_filled_where_pytorch_fills_them():
    # rows behind the batch are left as they were: in deterministic mode that is what torch.empty gives there
    need_cuda()
    from torch.utils.deterministic import fill_uninitialized_memory
    assert fill_uninitialized_memory
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(4, 4, 64, generator=g, device="cuda")
    kc, vc = (torch.randn(6, 2, 16, 64, generator=g, device="cuda") for _ in range(2))
    args = (q, kc, vc, i32([0, 1]), i32([[0, 1, 2]]), i32([40]))
    want, wl = rsa.prefix_attn(*args)
    mode = torch.are_deterministic_algorithms_enabled()
    try:
        torch.use_deterministic_algorithms(True)
        out, lse = rsa.prefix_attn(*args)
    finally:
        torch.use_deterministic_algorithms(mode)
    assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0])
    assert out[1:].isnan().all() and lse[1:].isnan().all()


def test_tensors_that_a_call_makes_are_seen_by_a_mode():
    need_cuda()
    from torch.utils._python_dispatch import TorchDispatchMode
    seen = []

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            r = func(*args, **(kwargs or {}))
            seen.append((func, tuple(r.shape) if isinstance(r, torch.Tensor) else None))
            return r
    args = step_of()
    with Seen():
        dq, dk, dwq, dwk = rsa.qk_norm_rope_bwd(*args)
    made = [s for f, s in seen if f is torch.ops.aten.empty.memory_format]
    for t in (dq, dk, dwq, dwk):
        assert tuple(t.shape) in made
    for x, y in zip((dq, dk, dwq, dwk), rsa.qk_norm_rope_bwd(*args)):
        assert torch.equal(x, y)
    rsa.check_device_error()
