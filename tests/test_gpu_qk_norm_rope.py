"""qk_norm_rope and its gradient on the GPU against the 64-bit forms."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

CASES = [
    # T, Hq, Hkv, d, rot, interleaved, sections, dtype
    (1, 1, 1, 128, 128, False, None, torch.bfloat16),
    (1, 64, 8, 128, 128, False, None, torch.bfloat16),
    (7, 5, 3, 128, 128, True, None, torch.bfloat16),
    (33, 9, 2, 64, 64, False, None, torch.bfloat16),
    (130, 3, 1, 64, 32, True, None, torch.bfloat16),
    (257, 4, 4, 128, 48, False, [5, 11, 8], torch.bfloat16),
    (65, 6, 2, 128, 112, True, [20, 0, 36], torch.bfloat16),
    (50, 2, 2, 64, 0, False, None, torch.bfloat16),
    (1, 8, 8, 64, 64, True, None, torch.float32),
    (19, 7, 1, 128, 128, False, None, torch.float32),
    (100, 4, 2, 64, 16, False, None, torch.float32),
    (77, 5, 5, 128, 96, True, [16, 16, 15, 1], torch.float32),
    (3001, 2, 1, 64, 64, False, [31, 1], torch.float32),
]
IDS = ["T{}q{}k{}d{}r{}{}{}{}".format(*c[:5], "i" if c[5] else "h", "" if c[6] is None else "x%d" % len(c[6]),
                                      "bf" if c[7] == torch.bfloat16 else "f") for c in CASES]


def make(case, seed=0, max_pos=4000):
    T, Hq, Hkv, d, rot, inter, sections, dt = case
    g = torch.Generator().manual_seed(seed)
    packed = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(dt).cuda()
    q = packed[:, :Hq * d].view(T, Hq, d)
    k = packed[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    v = packed[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    wq, wk = ((1 + 0.5 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(2))
    table = rsa.rope_table(max_pos, rot) if rot else None
    shape = (T,) if sections is None else (len(sections), T)
    pos = torch.randint(0, max_pos, shape, generator=g)
    pos.view(-1)[0], pos.view(-1)[-1] = max_pos - 1, 0
    return q, k, v, wq, wk, pos.cuda(), table


def reference(x, w, pos, table, case, eps):
    t = None if table is None else ref.to64(table)
    return ref.norm_rope(ref.to64(x), None if w is None else ref.to64(w), pos.cpu().numpy(), t, eps, case[5], case[6])


def close(got, want, bound, dtype, what):
    tol = bound + ref.half_step(dtype) * np.abs(want)
    worst = (np.abs(ref.to64(got) - want) / tol).max()
    assert worst <= 1, f"{what} is {worst:.3g} times its bound off"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    need_cuda()
    eps = 1e-5
    q, k, v, wq, wk, pos, table = make(case)
    qo, ko = rsa.qk_norm_rope(q, k, wq, wk, pos, table, eps=eps, interleaved=case[5], sections=case[6])
    torch.cuda.synchronize()
    rsa.check_device_error()
    close(qo, *reference(q, wq, pos, table, case, eps), case[7], "q")
    close(ko, *reference(k, wk, pos, table, case, eps), case[7], "k")
    # in place, and without weights
    q2, k2 = q.clone(), k.clone()
    a, b = rsa.qk_norm_rope(q2, k2, None, wk, pos, table, eps=eps, interleaved=case[5], sections=case[6], q_out=q2, k_out=k2)
    assert a is q2 and b is k2
    close(q2, *reference(q, None, pos, table, case, eps), case[7], "q in place")
    assert torch.equal(k2, ko)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("page", [16, 128])
def test_cache_write(case, page):
    need_cuda()
    T, Hq, Hkv, d, dt = case[0], case[1], case[2], case[3], case[7]
    q, k, v, wq, wk, pos, table = make(case, seed=1)
    n_pages = T // page + 3
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.randn(n_pages, Hkv, page, d, generator=g).to(dt).cuda() for _ in range(2))
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    if T > 1:
        slots[-1] = -(1 << 40)
    wk_c, wv_c = kc.clone(), vc.clone()
    kw = dict(interleaved=case[5], sections=case[6])
    qo, none = rsa.qk_norm_rope(q, k, wq, wk, pos, table, v=v, slot_map=slots.cuda(), k_cache=kc, v_cache=vc, **kw)
    assert none is None
    q1, k1 = rsa.qk_norm_rope(q, k, wq, wk, pos, table, **kw)  # held to the definition above
    live = slots >= 0
    at, row = slots[live] // page, slots[live] % page
    wk_c[at.cuda(), :, row.cuda()] = k1[live.cuda()]
    wv_c[at.cuda(), :, row.cuda()] = v[live.cuda()]
    torch.cuda.synchronize()
    rsa.check_device_error()
    assert torch.equal(qo, q1)
    assert torch.equal(kc, wk_c) and torch.equal(vc, wv_c)  # the other slots as they were
    ko = torch.empty_like(k1)
    rsa.qk_norm_rope(q, k, wq, wk, pos, table, v=v, slot_map=slots.cuda(), k_cache=kc, v_cache=vc, k_out=ko, **kw)
    assert torch.equal(ko, k1)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    need_cuda()
    T, Hq, Hkv, d, rot, inter, sections, dt = case
    eps = 1e-5
    q, k, v, wq, wk, pos, table = make(case, seed=2)
    g = torch.Generator().manual_seed(9)
    gq, gk = torch.randn(T, Hq, d, generator=g).to(dt).cuda(), torch.randn(T, Hkv, d, generator=g).to(dt).cuda()
    dq, dk, dwq, dwk = rsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, table, eps=eps, interleaved=inter, sections=sections)
    torch.cuda.synchronize()
    rsa.check_device_error()
    t = None if table is None else ref.to64(table)
    for name, dy, x, w, dx, dw in (("q", gq, q, wq, dq, dwq), ("k", gk, k, wk, dk, dwk)):
        rx, rw, bound, size = ref.norm_rope_bwd(ref.to64(dy), ref.to64(x), ref.to64(w), pos.cpu().numpy(), t, eps, inter, sections)
        close(dx, rx, bound, dt, "d" + name)
        # each term within 32 roundings; a chain of additions: a lane's own (at most all the rows of 8 heads of
        # its items), the block's 8 to 32 groups, 608 / 32 partial rows, 32 sums
        depth = 32 + T * x.shape[1] / min(608, T) + 32 + 19 + 32
        worst = (np.abs(ref.to64(dw) - rw) / (depth * ref.U32 * size)).max()
        assert worst <= 1, f"dw of {name} is {worst:.3g} times its bound off"
    # the same again bit for bit, in place, and with a weight that is not wanted
    a, b = gq.clone(), gk.clone()
    r = rsa.qk_norm_rope_bwd(a, b, q, k, wq, wk, pos, table, eps=eps, interleaved=inter, sections=sections, dq=a, dk=b)
    for x, y in zip(r, (dq, dk, dwq, dwk)):
        assert torch.equal(x, y)
    r = rsa.qk_norm_rope_bwd(gq, gk, q, k, None, wk, pos, table, eps=eps, interleaved=inter, sections=sections)
    assert r[2] is None and torch.equal(r[3], dwk) and torch.equal(r[1], dk)


def test_backward_against_differences():
    # the kernels' own forward, differenced along a random direction of x and of w (fp32: steps of 2^-9, second
    # order below 2^-18 of the third derivatives, rounding of the sums about 2^-24 / 2^-9 of their size)
    need_cuda()
    case = (40, 4, 2, 64, 64, False, None, torch.float32)
    q, k, v, wq, wk, pos, table = make(case, seed=3)
    g = torch.Generator().manual_seed(1)
    q, k = q.contiguous(), k.contiguous()
    gq, gk = torch.randn(q.shape, generator=g).cuda(), torch.randn(k.shape, generator=g).cuda()
    dq, dk, dwq, dwk = rsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, table)
    f = lambda q, k, wq, wk: sum((x.double() * y.double()).sum() for x, y in zip(rsa.qk_norm_rope(q, k, wq, wk, pos, table), (gq, gk)))  # noqa: E731
    h = 2.0 ** -9
    args = [q, k, wq, wk]
    for i, grad in enumerate((dq, dk, dwq, dwk)):
        e = torch.randn(grad.shape, generator=g).cuda()
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * e, args[i] - h * e
        num = float((f(*up) - f(*dn)) / (2 * h))
        ana = float((grad.double() * e.double()).sum())
        size = float((grad.double() * e.double()).norm()) + 1
        assert abs(num - ana) <= 2e-2 * size, (i, num, ana, size)


def test_special_values():
    need_cuda()
    d = 128
    table = rsa.rope_table(10, d)
    x = torch.zeros(4, 1, d, device="cuda")
    x[1] = 1e-30                      # squares vanish: eps alone
    x[2, 0, 5] = float("inf")
    x[3, 0, 7] = float("nan")
    k = torch.ones(4, 1, d, device="cuda")
    pos = torch.tensor([0, 3, 4, 5], device="cuda")
    qo, ko = rsa.qk_norm_rope(x, k, None, None, pos, table)
    assert torch.equal(qo[0], x[0])                       # a row of zeros stays zero
    assert torch.isfinite(qo[1]).all() and qo[1].abs().max() < 1e-26
    assert torch.isnan(qo[2]).any()                       # inf / inf in its own row
    assert torch.isnan(qo[3]).all()
    assert torch.isfinite(ko).all()                       # ... and in no other
    # eps 0 and a row of zeros: 0 * inf, as the formula has it
    qo, _ = rsa.qk_norm_rope(x[:1], k[:1], None, None, pos[:1], table, eps=0.0)
    assert torch.isnan(qo).all()
    rsa.check_device_error()


def test_positions_and_slots_out_of_range_are_reported_and_harmless():
    need_cuda()
    d, page = 64, 16
    table = rsa.rope_table(8, d)
    q, k, v = (torch.randn(5, 2, d, device="cuda") for _ in range(3))
    good = torch.tensor([0, 1, 2, 3, 4], device="cuda")
    want, wk = rsa.qk_norm_rope(q, k, None, None, good, table)
    for bad in (8, -1, 1 << 40):
        pos = good.clone()
        pos[2] = bad
        got, _ = rsa.qk_norm_rope(q, k, None, None, pos, table)
        with pytest.raises(rsa.RsaError) as e:
            rsa.check_device_error()
        assert e.value.status == 3
        keep = [0, 1, 3, 4]
        assert torch.equal(got[keep], want[keep])
    kc, vc = torch.zeros(3, 2, page, d, device="cuda"), torch.zeros(3, 2, page, d, device="cuda")
    slots = torch.tensor([0, 3 * page, 1 << 40, 5, 3 * page - 1], device="cuda")  # the second and third are not in the cache
    rsa.qk_norm_rope(q, k, None, None, good, table, v=v, slot_map=slots, k_cache=kc, v_cache=vc)
    with pytest.raises(rsa.RsaError):
        rsa.check_device_error()
    wkc, wvc = torch.zeros_like(kc), torch.zeros_like(vc)
    for t in (0, 3, 4):
        s = int(slots[t])
        wkc[s // page, :, s % page], wvc[s // page, :, s % page] = wk[t], v[t]
    assert torch.equal(kc, wkc) and torch.equal(vc, wvc)
    rsa.check_device_error()


def test_streams_strides_and_refusals():
    need_cuda()
    d = 64
    table = rsa.rope_table(100, d)
    base = torch.randn(3, 50, d, device="cuda")      # heads first: [H, T, d]
    q = base.transpose(0, 1)
    pos = torch.arange(50, device="cuda")
    want, _ = rsa.qk_norm_rope(q.contiguous(), q.contiguous(), None, None, pos, table)
    out = torch.empty(3, 50, d, device="cuda").transpose(0, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = rsa.qk_norm_rope(q, q, None, None, pos, table, q_out=out, stream=s)
    got2, _ = rsa.qk_norm_rope(q, q, None, None, pos, table, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)
    for bad in (dict(q_out=torch.empty(50, 2, d, device="cuda")), dict(k_out=torch.empty(50, 3, d, device="cuda").bfloat16()),
                dict(slot_map=pos), dict(v=q), dict(sections=[16, 16]), dict(sections=[31])):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            rsa.qk_norm_rope(q, q, None, None, pos, table, **bad)
    with pytest.raises(ValueError):
        rsa.qk_norm_rope(q, q, torch.ones(32, device="cuda"), None, pos, table)
    with pytest.raises(ValueError):
        rsa.qk_norm_rope(q, q, None, None, pos[:-1], table)
    with pytest.raises(TypeError):
        rsa.qk_norm_rope(q.half(), q.half(), None, None, pos, table)
    with pytest.raises(rsa.RsaError):  # a broadcast input: one row for all tokens
        rsa.qk_norm_rope(q[:1].expand(50, 3, d), q, None, None, pos, table)


def test_backward_captured():
    need_cuda()
    case = (100, 8, 2, 128, 128, False, None, torch.bfloat16)
    q, k, v, wq, wk, pos, table = make(case, seed=4)
    gq, gk = torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous())
    want = rsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = rsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, table)
    for _ in range(2):
        for x in got:
            x.zero_()
        g.replay()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
