"""Host-side checks of the paged-cache operators: refusals before anything is
launched, workspace sizes, and the tests' own 64-bit forms (a gradient against
differences, the plan by hand).  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from context_attention_rsa_gb300 import paged

FAKE = 0x100000  # aligned and never dereferenced
INVALID, UNSUPPORTED = 1, 2


def plan_call(**kw):
    a = dict(cached=0x100000, new=0x200000, R=4, page=64, n_pages=100, table=0x300000, stride=8, max_pages=8, free=0x400000,
             n_free=50, start=0x500000, pos0=0, max_tokens=128, cu=0x600000, kv=0x700000, slots=0x800000, pos=0x900000,
             info=0xa00000)
    a.update(kw)
    return rsa.load().rsa_page_plan(a["cached"], a["new"], a["R"], a["page"], a["n_pages"], a["table"], a["stride"],
                                    a["max_pages"], a["free"], a["n_free"], a["start"], a["pos0"], a["max_tokens"], a["cu"],
                                    a["kv"], a["slots"], a["pos"], a["info"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), INVALID), (dict(R=16385), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(stride=7), INVALID),
    (dict(max_pages=1 << 26, stride=1 << 26), INVALID),          # 2^32 own tokens
    (dict(n_free=-1), INVALID), (dict(n_free=1 << 31), INVALID), (dict(pos0=-1), INVALID), (dict(max_tokens=0), INVALID),
    (dict(max_tokens=1 << 31), INVALID), (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID),
    (dict(free=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(slots=None), INVALID),
    (dict(pos=None), INVALID), (dict(info=None), INVALID), (dict(cached=FAKE + 2), INVALID), (dict(slots=0x800008), INVALID),
    (dict(start=0x500004), INVALID),
    (dict(kv=0x100000), INVALID),       # kv_len over cached_len
    (dict(kv=0x10000c), INVALID),       # overlapping by one entry
    (dict(start=0xa00018), INVALID),    # free_start inside info
    (dict(pos=0x8003f8), INVALID),      # misaligned and overlapping
    (dict(pos=0x8003f0), INVALID),      # positions over the end of slot_map
])
def test_page_plan_refuses(kw, code):
    assert plan_call(**kw) == code, rsa.load().rsa_last_error_string()


def rope_args(**kw):
    a = paged.NormRopeArgs()
    a.dt, a.T, a.Hq, a.Hkv, a.d = 1, 10, 8, 2, 128
    a.q, a.k = paged.Heads(FAKE, 12 * 128, 128), paged.Heads(FAKE, 12 * 128, 128)
    a.eps, a.rot, a.n_axes = 1e-6, 128, 1
    a.positions, a.cos_sin, a.max_pos = FAKE, FAKE, 100
    for name, v in kw.items():
        if name == "sections":
            a.sections[:len(v)] = v
        else:
            setattr(a, name, v)
    return a


BAD_ROPE = [
    (dict(dt=2), INVALID), (dict(T=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(rot=8), INVALID), (dict(rot=144), INVALID), (dict(rot=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID), (dict(n_axes=2, sections=(32, 31)), INVALID),
    (dict(n_axes=2, sections=(65, -1)), INVALID), (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID),
    (dict(cos_sin=FAKE + 8), INVALID), (dict(max_pos=0), INVALID), (dict(q=paged.Heads(None, 1024, 128)), INVALID),
    (dict(q=paged.Heads(FAKE + 8, 1024, 128)), INVALID), (dict(q=paged.Heads(FAKE, 1020, 128)), INVALID),
    (dict(k=paged.Heads(FAKE, 0, 128)), INVALID), (dict(k=paged.Heads(FAKE, 1024, 64)), INVALID),
    (dict(q_weight=FAKE + 4), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_ROPE)
def test_qk_norm_rope_refuses(kw, code):
    lib = rsa.load()
    out, ko, none = paged.Heads(FAKE, 1024, 128), paged.Heads(FAKE, 256, 128), paged.Heads()
    a = rope_args(**kw)
    assert lib.rsa_qk_norm_rope_fwd(ctypes.byref(a), out, ko, none, None, None, None, 0, 0, None) == code
    assert lib.rsa_qk_norm_rope_bwd(ctypes.byref(a), out, ko, out, ko, FAKE, FAKE, FAKE, 1 << 30, None) == code


def test_qk_norm_rope_refuses_bad_results_and_caches():
    lib = rsa.load()
    a = ctypes.byref(rope_args())
    out, ko, v = paged.Heads(FAKE, 1024, 128), paged.Heads(FAKE, 256, 128), paged.Heads(FAKE, 1536, 128)
    none = paged.Heads()

    def fwd(out=out, ko=ko, v=v, slots=FAKE, kc=FAKE, vc=FAKE, page=64, n=10):
        return lib.rsa_qk_norm_rope_fwd(a, out, ko, v, slots, kc, vc, page, n, None)
    assert lib.rsa_qk_norm_rope_fwd(None, out, ko, v, FAKE, FAKE, FAKE, 64, 10, None) == INVALID
    assert fwd(out=none) == INVALID
    assert fwd(ko=none, slots=None) == INVALID                      # k has to go somewhere
    assert fwd(out=paged.Heads(FAKE, 128, 128)) == INVALID          # rows of several tokens on one another
    assert b"overlapping" in lib.rsa_last_error_string()
    assert fwd(v=none) == INVALID
    assert fwd(slots=FAKE + 4) == INVALID
    assert fwd(kc=None) == INVALID and fwd(vc=FAKE + 2) == INVALID
    assert fwd(page=24) == UNSUPPORTED and fwd(n=0) == INVALID and fwd(n=1 << 30, page=16) == INVALID  # 2^31 page heads
    n = ctypes.c_size_t(0)
    assert lib.rsa_qk_norm_rope_bwd_workspace_size(128, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.rsa_qk_norm_rope_bwd_workspace_size(80, ctypes.byref(n)) == UNSUPPORTED
    assert lib.rsa_qk_norm_rope_bwd_workspace_size(128, None) == INVALID

    def bwd(gq=out, gk=ko, dq=out, dk=ko, ws=FAKE, nb=1 << 30):
        return lib.rsa_qk_norm_rope_bwd(a, gq, gk, dq, dk, FAKE, None, ws, nb, None)
    assert bwd(gq=none) == INVALID and bwd(gk=none) == INVALID and bwd(dq=none) == INVALID and bwd(dk=none) == INVALID
    assert bwd(ws=None) == INVALID and bwd(ws=FAKE + 4) == INVALID
    assert bwd(nb=n.value - 1) == INVALID and b"needed" in lib.rsa_last_error_string()
    assert bwd(dk=paged.Heads(FAKE, 128, 128)) == INVALID


def attn_call(**kw):
    a = dict(q=FAKE, qt=1024, qh=128, kc=FAKE, vc=FAKE, dt=1, T=16, Hq=8, Hkv=2, d=128, page=64, n_pages=100, cu=FAKE, kv=FAKE,
             R=4, table=FAKE, stride=8, max_pages=8, pp=FAKE, plen=100, out=FAKE, lse=FAKE, ws=FAKE, nb=1 << 40)
    a.update(kw)
    return rsa.load().rsa_prefix_attn_fwd(a["q"], a["qt"], a["qh"], a["kc"], a["vc"], a["dt"], a["T"], a["Hq"], a["Hkv"],
                                          a["d"], a["page"], a["n_pages"], a["cu"], a["kv"], a["R"], a["table"], a["stride"],
                                          a["max_pages"], a["pp"], a["plen"], a["out"], a["lse"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), INVALID), (dict(T=0), INVALID), (dict(R=0), INVALID), (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=100), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(n_pages=1 << 30), INVALID),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qt=4), INVALID), (dict(qt=1028), INVALID), (dict(qh=0), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(stride=7), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 25, stride=1 << 25), INVALID), (dict(plen=-1), INVALID),
    (dict(plen=1 << 31), INVALID), (dict(pp=None), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 4), INVALID),
    (dict(nb=1000), INVALID),
])
def test_prefix_attn_refuses(kw, code):
    assert attn_call(**kw) == code, rsa.load().rsa_last_error_string()


# addresses far enough apart for the shape above: 1024 bytes a token of q, 16 KB of cache a page and key head
APART = dict(q=0x1000000, kc=0x2000000, vc=0x3000000, out=0x4000000, lse=0x5000000, ws=0x10000000, nb=0x10000000)


@pytest.mark.parametrize("kw,what", [
    (dict(out=0x1000000), b"out overlaps q"), (dict(out=0x1000000 + 15 * 2048), b"out overlaps q"),
    (dict(out=0x2000000 + 100 * 2 * 64 * 128 * 2 - 16), b"out overlaps k_cache"), (dict(lse=0x3000010), b"lse overlaps v_cache"),
    (dict(lse=0x4000010), b"lse overlaps out"), (dict(ws=0x4000000 - 0x1000000), b"workspace overlaps"),
    (dict(ws=0x800000), b"workspace overlaps q"),
    (dict(plen=(1 << 31) - 127), b"prefix_len"), (dict(plen=(1 << 31) - 1), b"prefix_len"),
    (dict(R=(1 << 30) + 1, nb=1 << 40, ws=1 << 41), b"requests"),
])
def test_prefix_attn_refuses_overlaps_and_lengths_that_do_not_fit(kw, what):
    code = attn_call(**{**APART, **kw})
    assert code in (INVALID, UNSUPPORTED) and what in rsa.load().rsa_last_error_string(), rsa.load().rsa_last_error_string()


def test_prefix_attn_workspace_size():
    # a plan, two homes for every row, 256 rows for each of 160 workers; no term in the lengths
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    T, Hq, Hkv, d, R = 17, 40, 8, 128, 9
    want = up((R + 3) * 8) + 2 * (up(T * Hq * d * 4) + up(T * Hq * 4)) + up(160 * 256 * d * 4) + up(160 * 256 * 4)
    assert rsa.prefix_attn_workspace_size(torch.bfloat16, T, Hq, Hkv, d, R) == want
    with pytest.raises(rsa.RsaError) as e:
        rsa.prefix_attn_workspace_size(torch.float16, T, Hq, Hkv, d, R)
    assert e.value.status == INVALID
    with pytest.raises(rsa.RsaError):
        rsa.prefix_attn_workspace_size(torch.bfloat16, T, 41, Hkv, d, R)


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError):
        rsa.qk_norm_rope(x, x, None, None, torch.zeros(4, dtype=torch.int64), None)
    with pytest.raises(TypeError):
        rsa.prefix_attn(x, x, x, x, x, x)
    with pytest.raises(TypeError):
        rsa.page_plan(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2), x, 16, 4, 8)


def test_reference_gradient_against_differences():
    # the formulas that the backward kernel is held to, against central differences of the forward's definition
    rng = np.random.default_rng(0)
    T, H, d, eps = 2, 3, 64, 1e-3
    x, dy, w = rng.standard_normal((T, H, d)), rng.standard_normal((T, H, d)), 1 + 0.3 * rng.standard_normal(d)
    pos = rng.integers(0, 50, (2, T))
    table = rsa.rope_table(50, 48, device="cpu").double().numpy()
    for inter in (False, True):
        f = lambda x, w: (dy * ref.norm_rope(x, w, pos, table, eps, inter, [10, 14])[0]).sum()  # noqa: E731
        dx, dw, _, _ = ref.norm_rope_bwd(dy, x, w, pos, table, eps, inter, [10, 14])
        h = 1e-5
        for i in [(0, 0, 0), (0, 1, 13), (1, 2, 40), (1, 0, 63)]:
            e = np.zeros_like(x)
            e[i] = h
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
        for i in (0, 13, 47, 63):
            e = np.zeros(d)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_rope_table_keeps_far_angles():
    t = rsa.rope_table(1 << 20, 64, device="cpu")
    import math
    for pos in (0, 1, 65537, (1 << 20) - 1):
        for i in (0, 7, 31):
            a = pos * 10000.0 ** (-2 * i / 64)
            assert abs(float(t[pos, i]) - math.cos(a)) < 1e-7 and abs(float(t[pos, 32 + i]) - math.sin(a)) < 1e-7


def test_reference_plan_by_hand():
    table = np.full((2, 3), -1, np.int32)
    table[0, 0] = 5
    t, cu, kv, slots, pos, info = ref.page_plan([3, 0], [2, 1], table, [9, 8, 7], 4, 5, start=1, pos0=10)
    assert t.tolist() == [[5, 8, -1], [7, -1, -1]] and cu.tolist() == [0, 2, 3] and kv.tolist() == [5, 1]
    assert slots.tolist() == [23, 32, 28, -1, -1] and pos.tolist() == [13, 14, 10, 0, 0] and info.tolist() == [0, 3, 2, 3]
