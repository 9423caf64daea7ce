"""Host-side checks of the calls for drafted tokens and the keeping of pages: refusals
before anything is launched, operands that share memory, and the tests' own
plain forms by hand.  No GPU: every call is refused or stops before its launch."""
import ctypes

import numpy as np
import pytest
import torch

import drafts_reference as dr
import context_attention_rsa_gb300 as rsa
from context_attention_rsa_gb300 import paged

INVALID, UNSUPPORTED, STOPPED = 1, 2, 3


def stopped(call):
    """The status and text of a call whose launch is not made."""
    lib = rsa.load()
    lib.rsa_debug_inject_launch_failure(0)
    try:
        return call(lib), lib.rsa_last_error_string()
    finally:
        lib.rsa_debug_inject_launch_failure(-1)


# ---- tree_plan -------------------------------------------------------------------------

def plan_call(**kw):
    a = dict(parent=0x100000, T=16, cu=0x200000, kv=0x300000, R=4, words=2, pos0=0, pos=0x400000, mask=0x500000)
    a.update(kw)
    return stopped(lambda lib: lib.rsa_tree_plan(a["parent"], a["T"], a["cu"], a["kv"], a["R"], a["words"], a["pos0"], a["pos"],
                                                 a["mask"], None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INVALID), (dict(R=0), INVALID), (dict(words=0), INVALID), (dict(words=33), INVALID), (dict(pos0=-1), INVALID),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(R=(1 << 30) + 1), UNSUPPORTED),
    (dict(parent=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(pos=None), INVALID),
    (dict(mask=None), INVALID), (dict(parent=0x100002), INVALID), (dict(pos=0x400004), INVALID), (dict(mask=0x500002), INVALID),
    (dict(pos=0x100038), INVALID), (dict(mask=0x20000c), INVALID), (dict(mask=0x300000), INVALID), (dict(mask=0x400078), INVALID),
])
def test_tree_plan_refuses(kw, code):
    assert plan_call(**kw)[0] == code, kw


def test_tree_plan_takes_what_it_should():
    for kw in (dict(), dict(T=1, R=1, words=1), dict(words=32), dict(mask=0x200000 + 20), dict(pos=0x100040)):
        st, text = plan_call(**kw)
        assert st == STOPPED, (kw, text)


# ---- tree_attn -------------------------------------------------------------------------

def attn_call(**kw):
    a = dict(q=0x1000000, qt=1024, qh=128, kc=0x2000000, vc=0x3000000, dt=1, T=16, Hq=8, Hkv=2, d=128, page=64, n_pages=100, cu=0x100000,
             kv=0x100000, R=4, table=0x100000, stride=8, max_pages=8, pp=0x100000, plen=100, mask=0x200000, ms=2, words=2, out=0x4000000,
             lse=0x5000000, ws=0x10000000, nb=0x10000000)
    a.update(kw)
    return stopped(lambda lib: lib.rsa_tree_attn_fwd(
        a["q"], a["qt"], a["qh"], a["kc"], a["vc"], a["dt"], a["T"], a["Hq"], a["Hkv"], a["d"], a["page"], a["n_pages"], a["cu"], a["kv"],
        a["R"], a["table"], a["stride"], a["max_pages"], a["pp"], a["plen"], a["mask"], a["ms"], a["words"], a["out"], a["lse"], a["ws"],
        a["nb"], None))


@pytest.mark.parametrize("kw,code,what", [
    (dict(mask=None), INVALID, b"mask"), (dict(mask=0x200002), INVALID, b"mask"), (dict(words=0), INVALID, b"words"),
    (dict(words=33, ms=33), INVALID, b"words"), (dict(ms=1), INVALID, b"mask_stride"), (dict(ms=(1 << 30) + 1), INVALID, b"mask_stride"),
    (dict(out=0x200000 - 0x100), INVALID, b"out overlaps"), (dict(lse=0x200040), INVALID, b"lse overlaps mask"),
    (dict(ws=0x1ff000), INVALID, b"workspace overlaps"),
    # and all that prefix_attn refuses
    (dict(dt=5), INVALID, b""), (dict(T=0), INVALID, b""), (dict(Hq=9), INVALID, b""), (dict(d=256), UNSUPPORTED, b""),
    (dict(Hq=258), UNSUPPORTED, b""), (dict(page=8), UNSUPPORTED, b""), (dict(n_pages=0), INVALID, b""), (dict(q=None), INVALID, b""),
    (dict(qt=1028), INVALID, b""), (dict(table=None), INVALID, b""), (dict(stride=7), INVALID, b""), (dict(plen=-1), INVALID, b""),
    (dict(pp=None), INVALID, b""), (dict(nb=1000), INVALID, b"needed"), (dict(out=0x1000000), INVALID, b"out overlaps q"),
    (dict(lse=0x4000010), INVALID, b"lse overlaps out"),
])
def test_tree_attn_refuses(kw, code, what):
    st, text = attn_call(**kw)
    assert st == code and what in text, (st, text)


def test_tree_attn_workspace_size():
    # prefix_attn's, the sums of the pairs of token groups, and room to begin on 256 bytes
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for T, Hq, Hkv, d, R in ((17, 40, 8, 128, 9), (1, 1, 1, 64, 1), (1000, 64, 8, 64, 500)):
        want = rsa.prefix_attn_workspace_size(torch.bfloat16, T, Hq, Hkv, d, R) + up((R + 2) * 8) + 256
        assert rsa.tree_attn_workspace_size(torch.bfloat16, T, Hq, Hkv, d, R) == want
        shape = dict(T=T, Hq=Hq, Hkv=Hkv, d=d, R=R, qt=Hq * d, qh=d, q=1 << 40, kc=2 << 40, vc=3 << 40, out=4 << 40, lse=5 << 40, ws=6 << 40,
                     mask=7 << 40, plen=0)
        assert attn_call(**shape, nb=want - 1)[0] == INVALID and attn_call(**shape, nb=want)[0] == STOPPED
    with pytest.raises(rsa.RsaError):
        rsa.tree_attn_workspace_size(torch.float16, 1, 1, 1, 64, 1)
    assert rsa.load().rsa_tree_attn_workspace_size(1, 1, 1, 1, 64, 1, None) == INVALID


# ---- the caches' layers ------------------------------------------------------------------

LAYERS, PAGES, HKV, PAGE, D = 3, 50, 2, 64, 128
CACHE = LAYERS * PAGES * HKV * PAGE * D * 2
AT = dict(k=0x10000000, v=0x20000000, table=0x100000, cached=0x200000, kv=0x300000, keep=0x400000, keep_len=0x500000, out=0x600000,
          src=0x700000, dst=0x800000, free=0x900000, start=0xa00000, shares=0xb00000, info=0xc00000)


def cache(a):
    c = paged.Cache()
    c.k_cache, c.v_cache, c.dt, c.layers, c.n_pages = a["k"], a["v"], a.get("dt", 1), a.get("layers", LAYERS), a.get("n_pages", PAGES)
    c.Hkv, c.page_size, c.d = a.get("Hkv", HKV), a.get("page", PAGE), a.get("d", D)
    return None if a.get("null") else ctypes.byref(c)


BAD_CACHE = [
    (dict(null=True), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=0x10000008), INVALID), (dict(dt=2), INVALID),
    (dict(layers=0), INVALID), (dict(Hkv=0), INVALID), (dict(n_pages=0), INVALID), (dict(page=48), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(layers=32768, Hkv=1), UNSUPPORTED), (dict(n_pages=1 << 30, Hkv=2), INVALID), (dict(v=0x10000000 + CACHE - 16), INVALID),
    (dict(table=0x10000000), INVALID), (dict(table=None), INVALID), (dict(stride=7), INVALID), (dict(stride=1 << 31), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 25, stride=1 << 25), INVALID), (dict(R=0), INVALID),
]


def compact_call(**kw):
    a = {**AT, "R": 4, "stride": 8, "max_pages": 8, "ks": 6, "max_keep": 6, **kw}
    return stopped(lambda lib: lib.rsa_cache_compact(cache(a), a["table"], a["stride"], a["max_pages"], a["cached"], a["kv"], a["R"],
                                                     a["keep"], a["ks"], a["max_keep"], a["keep_len"], a["out"], None))


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(max_keep=0), INVALID), (dict(ks=5), INVALID), (dict(ks=1 << 31), INVALID), (dict(cached=None), INVALID), (dict(kv=None), INVALID),
    (dict(keep=None), INVALID), (dict(keep_len=None), INVALID), (dict(out=None), INVALID), (dict(out=0x600002), INVALID),
    (dict(out=0x200000), INVALID), (dict(out=0x30000c), INVALID), (dict(out=0x400000 + 5 * 4), INVALID),
    (dict(out=0x500008), INVALID), (dict(keep=0x20000000 + CACHE - 4), INVALID), (dict(out=0x10000000), INVALID),
])
def test_cache_compact_refuses(kw, code):
    st, text = compact_call(**kw)
    assert st == code, (kw, text)


def fork_call(**kw):
    a = {**AT, "R": 4, "stride": 8, "max_pages": 8, "F": 2, "n_free": 20, **kw}
    return stopped(lambda lib: lib.rsa_page_fork(cache(a), a["table"], a["stride"], a["max_pages"], a["kv"], a["R"], a["src"], a["dst"], a["F"],
                                                 a["free"], a["n_free"], a["start"], a["shares"], a["info"], None))


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(R=16385, F=1), UNSUPPORTED), (dict(F=0), INVALID), (dict(F=5), INVALID), (dict(n_free=-1), INVALID), (dict(n_free=1 << 31), INVALID),
    (dict(F=4, max_pages=1 << 24, stride=1 << 24, R=16000, page=16), INVALID),   # the table is over the caches
    (dict(kv=None), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(free=None), INVALID), (dict(info=None), INVALID),
    (dict(start=0xa00004), INVALID), (dict(info=0xc00004), INVALID), (dict(shares=0xb00002), INVALID),
    (dict(kv=0x700004), INVALID), (dict(dst=0x300000), INVALID), (dict(free=0x100000), INVALID), (dict(shares=0x900000), INVALID),
    (dict(info=0xa00000), INVALID), (dict(start=0xc00018), INVALID), (dict(shares=0x300000), INVALID), (dict(info=0x10000000), INVALID),
])
def test_page_fork_refuses(kw, code):
    st, text = fork_call(**kw)
    assert st == code, (kw, text)


def free_call(**kw):
    a = {**AT, "R": 4, "stride": 8, "max_pages": 8, "page": PAGE, "n_pages": PAGES, "n_free": 20, **kw}
    return stopped(lambda lib: lib.rsa_page_free(a["table"], a["stride"], a["max_pages"], a["kv"], a["keep_len"], a["R"], a["page"],
                                                 a["n_pages"], a["free"], a["n_free"], a["start"], a["shares"], a["info"], None))


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), INVALID), (dict(R=16385), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(n_pages=(1 << 23) + 1), UNSUPPORTED), (dict(table=None), INVALID), (dict(stride=7), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 25, stride=1 << 25), INVALID), (dict(kv=None), INVALID), (dict(keep_len=None), INVALID), (dict(free=None), INVALID),
    (dict(n_free=0), INVALID), (dict(n_free=1 << 31), INVALID), (dict(start=None), INVALID), (dict(start=0xa00004), INVALID),
    (dict(info=None), INVALID), (dict(shares=0xb00002), INVALID),
    (dict(free=0x100000), INVALID), (dict(free=0x300004), INVALID), (dict(free=0x50000c), INVALID), (dict(free=0xa00000), INVALID),
    (dict(shares=0x900000 + 19 * 4), INVALID), (dict(info=0x900000), INVALID), (dict(info=0xa00000), INVALID), (dict(shares=0xc00018), INVALID),
])
def test_page_free_refuses(kw, code):
    st, text = free_call(**kw)
    assert st == code, (kw, text)


def test_calls_that_fit_reach_their_launch():
    # (without a GPU they stop where they ask for the device, a step before the launch)
    for call, kws in (
            (attn_call, (dict(), dict(plen=0, pp=None), dict(T=1, ms=1, words=1), dict(ms=1 << 10))),
            (compact_call, (dict(), dict(dt=0, d=64), dict(layers=1, max_keep=1, ks=1, R=1))),
            (fork_call, (dict(), dict(start=None), dict(shares=None), dict(n_free=0, free=None), dict(F=4))),
            (free_call, (dict(), dict(shares=None), dict(n_free=1), dict(n_pages=1 << 23, shares=None)))):
        for kw in kws:
            st, text = call(**kw)
            assert st == STOPPED, (kw, st, text)


def test_python_calls_refuse_host_tensors():
    x, i = torch.zeros(4, 2, 16, 64), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: rsa.tree_plan(i, i, i, 4), lambda: rsa.tree_attn(x[0], x, x, i, i, i, i),
                 lambda: rsa.cache_compact(x, x, i, i, i, i, i), lambda: rsa.page_fork(x, x, i, i, i, i, i),
                 lambda: rsa.page_free(i, i, i, i, i, 16, 4)):
        with pytest.raises(TypeError):
            call()


# ---- the plain forms, by hand --------------------------------------------------------------

def test_plain_tree_plan_by_hand():
    pos, mask = dr.tree_plan([-1, 0, 0, 1, -1], [0, 4, 5], [14, 3], 1, 6, pos0=100)
    assert pos.tolist() == [110, 111, 111, 112, 102, 0]
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b1, 0]


def test_plain_page_keeping_by_hand():
    page = 4
    caches = [np.arange(6 * page).reshape(1, 6, 1, page, 1).astype(float)]
    table = np.array([[3, 1], [0, 0]], np.int32)
    new, lens = dr.compact(caches, table, [1], [[1, 4]], [2], page)         # rows 1, 2 take rows 2 and 5
    assert new[0][0, 3, 0, :, 0].tolist() == [12, 14, 5, 15] and lens == [3]
    c, t, kv, sh, info = dr.fork(caches, table, [6, 0], [0], [1], [9, 5], 1, np.zeros(6, np.int32), page)
    assert t.tolist() == [[3, 1], [3, 5]] and kv == [6, 6] and sh.tolist() == [0, 0, 0, 1, 0, 0] and info == [0, 1, 1, 2]
    assert c[0][0, 5, 0, :, 0].tolist() == [4, 5, 22, 23]
    free, sh, info = dr.free_pages(t, [6, 6], [0, 0], np.array([7, 7, 7, 7]), 3, sh, page, 6)
    assert free.tolist() == [1, 3, 5, 7] and sh.tolist() == [0] * 6 and info == [0, 3, 4, 0]


@pytest.mark.parametrize("R,max_pages,code", [(16384, 1 << 16, None), (16384, (1 << 16) + 1, UNSUPPORTED), (8192, 1 << 17, None),
                                              (16384, (1 << 17) - 1, UNSUPPORTED)])
def test_entries_of_a_page_free(R, max_pages, code):
    # (a table of up to 8 GB, and what else there is behind it)
    at = {k: v + (1 << 40) for k, v in AT.items() if k != "table"}
    st, text = free_call(R=R, max_pages=max_pages, stride=max_pages, page=16, **at)
    assert st == (code or STOPPED), text


@pytest.mark.parametrize("max_keep,code", [(1 << 30, None), ((1 << 30) + 1, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)])
def test_longest_list_of_a_compaction(max_keep, code):
    st, text = compact_call(R=1, max_keep=max_keep, ks=max_keep, keep=1 << 40)
    assert st == (code or STOPPED), text
