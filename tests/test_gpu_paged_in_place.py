"""The head norm and its gradient in place: results on their inputs' own rows, in the
packed buffer that q, k and v are cut from, over several items a group of lanes."""
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf", "f"])


def cut(x, Hq, Hkv, d, turns):
    """q, k and v of packed rows: one after the other, or (Hq = Hkv) head by head in turn."""
    T = x.shape[0]
    if turns:
        y = x.view(T, Hq, 3, d)
        return y[:, :, 0], y[:, :, 1], y[:, :, 2]
    return x[:, :Hq * d].view(T, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d), x[:, (Hq + Hkv) * d:].view(T, Hkv, d)


@DTYPES
@pytest.mark.parametrize("T,Hq,Hkv,d,turns", [(1, 8, 8, 64, True), (1, 5, 2, 128, False), (6000, 8, 2, 128, False),
                                              (6000, 6, 6, 64, True)])
def test_forward_in_the_projection(dtype, T, Hq, Hkv, d, turns):
    need_cuda()
    page = 32
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g, device="cuda").to(dtype)
    pos, table = torch.arange(T, device="cuda"), rsa.rope_table(T, d)
    n_pages = -(-T // page)
    q, k, v = (t.contiguous() for t in cut(x, Hq, Hkv, d, turns))
    want = [torch.zeros(n_pages, Hkv, page, d, device="cuda", dtype=dtype) for _ in range(2)]
    wk = torch.empty_like(k)
    wq, _ = rsa.qk_norm_rope(q, k, None, None, pos, table, v=v, slot_map=pos, k_cache=want[0], v_cache=want[1], k_out=wk)
    got = [torch.zeros_like(want[0]) for _ in range(2)]
    q, k, v = cut(x, Hq, Hkv, d, turns)
    before = v.clone()
    rsa.qk_norm_rope(q, k, None, None, pos, table, v=v, slot_map=pos, k_cache=got[0], v_cache=got[1], q_out=q, k_out=k)
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(v, before)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rsa.check_device_error()


@DTYPES
@pytest.mark.parametrize("T,Hq,Hkv,d,turns", [(1, 3, 3, 64, True), (6000, 8, 2, 128, False), (6000, 6, 6, 64, True)])
def test_gradient_over_the_projection_or_over_its_own_gradient(dtype, T, Hq, Hkv, d, turns):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x, dy = (torch.randn(T, (Hq + 2 * Hkv) * d, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    pos, table = torch.arange(T, device="cuda"), rsa.rope_table(T, d)

    def run(x, dy, **kw):
        (q, k, _), (gq, gk, _) = cut(x, Hq, Hkv, d, turns), cut(dy, Hq, Hkv, d, turns)
        places = dict(x=(q, k), dy=(gq, gk))
        out = {"d" + n: places[p][n == "k"] for n, p in kw.items()}
        return rsa.qk_norm_rope_bwd(gq, gk, q, k, *w, pos, table, **out)
    want = run(x, dy)
    for kw in (dict(q="x", k="x"), dict(q="dy", k="dy"), dict(q="x", k="dy")):
        got = run(x.clone(), dy.clone(), **kw)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    rsa.check_device_error()


def test_tied_keys_and_values_in_place_are_refused():
    need_cuda()
    x = torch.randn(40, 16, 64, device="cuda")
    caches = [torch.zeros(3, 16, 16, 64, device="cuda") for _ in range(2)]
    t = torch.arange(40, device="cuda")
    with pytest.raises(rsa.RsaError) as e:
        rsa.qk_norm_rope(x.clone(), x, None, None, None, None, v=x, slot_map=t, k_cache=caches[0], v_cache=caches[1], k_out=x)
    assert e.value.status == 1 and "k_out overlaps v" in str(e.value)
    rsa.qk_norm_rope(x.clone(), x, None, None, None, None, v=x, slot_map=t, k_cache=caches[0], v_cache=caches[1])
    assert torch.equal(caches[1].transpose(1, 2).reshape(48, 16, 64)[:40], x)
    rsa.check_device_error()
