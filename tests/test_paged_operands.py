"""Operands of the paged-cache calls that share memory: what would be read after
it has been written is refused, rows of one packed buffer are not.  Host side
only: every call either is refused or stops before its launch (a failure is
injected there), so that addresses are never used, with a GPU or without."""
import ctypes

import numpy as np
import pytest
import torch

import context_attention_rsa_gb300 as rsa
from context_attention_rsa_gb300 import paged

INVALID, STOPPED = 1, 3
T, HQ, HKV, D, PAGE, PAGES = 10, 8, 2, 128, 16, 5
ROW = 2 * D                                   # bytes of a bf16 row
CACHE = PAGES * HKV * PAGE * ROW
# far enough apart for the shapes above
AT = dict(q=0x1000000, k=0x2000000, v=0x3000000, q_out=0x4000000, k_out=0x5000000, k_cache=0x6000000, v_cache=0x7000000,
          q_weight=0x8000000, k_weight=0x8100000, positions=0x8200000, cos_sin=0x8300000, slot_map=0x8400000, dq_out=0x9000000,
          dk_out=0xa000000, dq=0xb000000, dk=0xc000000, dq_weight=0xd000000, dk_weight=0xd100000, workspace=0xe000000)


def stopped(call):
    """The status and text of a call whose launch is not made."""
    lib = rsa.load()
    lib.rsa_debug_inject_launch_failure(0)
    try:
        return call(lib), lib.rsa_last_error_string()
    finally:
        lib.rsa_debug_inject_launch_failure(-1)


def heads(at, H, strides):
    if isinstance(at, paged.Heads):
        return at
    return paged.Heads(at, *(strides or (H * D, D)))


def arguments(a, strides):
    r = paged.NormRopeArgs()
    r.dt, r.T, r.Hq, r.Hkv, r.d = 1, a.get("T", T), a.get("Hq", HQ), a.get("Hkv", HKV), D
    r.q, r.k = heads(a["q"], r.Hq, strides.get("q")), heads(a["k"], r.Hkv, strides.get("k"))
    r.q_weight, r.k_weight, r.positions, r.cos_sin = a["q_weight"], a["k_weight"], a["positions"], a["cos_sin"]
    r.eps, r.rot, r.n_axes, r.max_pos = 1e-6, D, 1, 100
    return r


def forward(strides={}, **kw):
    a = {**AT, **kw}
    r = arguments(a, strides)
    h = lambda n, H: heads(a[n], H, strides.get(n))  # noqa: E731
    return stopped(lambda lib: lib.rsa_qk_norm_rope_fwd(ctypes.byref(r), h("q_out", r.Hq), h("k_out", r.Hkv), h("v", r.Hkv),
                                                        a["slot_map"], a["k_cache"], a["v_cache"], PAGE, PAGES, None))


def backward(strides={}, **kw):
    a = {**AT, **kw}
    r = arguments(a, strides)
    h = lambda n, H: heads(a[n], H, strides.get(n))  # noqa: E731
    return stopped(lambda lib: lib.rsa_qk_norm_rope_bwd(ctypes.byref(r), h("dq_out", r.Hq), h("dk_out", r.Hkv), h("dq", r.Hq),
                                                        h("dk", r.Hkv), a["dq_weight"], a["dk_weight"], a["workspace"], 1 << 30,
                                                        None))


def test_operands_of_their_own_are_taken():
    assert forward()[0] == STOPPED and backward()[0] == STOPPED
    assert forward(slot_map=None, v=0, k_cache=0, v_cache=0)[0] == STOPPED
    assert forward(k_out=paged.Heads())[0] == STOPPED
    assert forward(v=AT["k"])[0] == STOPPED                 # tied keys and values, only read
    # the memory of what a call does not use may lie anywhere
    assert forward(slot_map=None, k_cache=AT["q"], v_cache=AT["q"], v=AT["q_out"])[0] == STOPPED
    assert backward(dq_weight=None, dk_weight=None)[0] == STOPPED


def test_results_exactly_on_their_inputs_are_taken():
    packed = ((HQ + 2 * HKV) * D, D)
    q, k, v = AT["q"], AT["q"] + HQ * ROW, AT["q"] + (HQ + HKV) * ROW
    cut = dict(q=packed, k=packed, v=packed)
    assert forward(q_out=AT["q"], k_out=AT["k"])[0] == STOPPED
    # q, k and v cut from one projection, in place; and with results cut from another one
    assert forward({**cut, "q_out": packed, "k_out": packed}, q=q, k=k, v=v, q_out=q, k_out=k)[0] == STOPPED
    assert forward({**cut, "q_out": packed, "k_out": packed}, q=q, k=k, v=v, k_out=AT["q_out"] + HQ * ROW)[0] == STOPPED
    for dq in ("q", "dq_out"):
        for dk in ("k", "dk_out"):
            assert backward(dq=AT[dq], dk=AT[dk])[0] == STOPPED
    # one token, whose stride says nothing; heads of q, k and v in turn
    assert forward({"q": (HQ * D, D), "q_out": (5 * D * HQ, D)}, T=1, q_out=AT["q"])[0] == STOPPED
    turns = (3 * 4 * D, 3 * D)
    three = {n: turns for n in ("q", "k", "v", "q_out", "k_out")}
    at = dict(q=AT["q"], k=AT["q"] + ROW, v=AT["q"] + 2 * ROW, q_out=AT["q"], k_out=AT["q"] + ROW, Hq=4, Hkv=4)
    assert forward(three, **at)[0] == STOPPED


@pytest.mark.parametrize("kw,what", [
    (dict(k_out="k", v="k"), "k_out overlaps v"),                       # tied keys and values, keys in place
    (dict(q_out="k"), "q_out overlaps k"), (dict(q_out="v"), "q_out overlaps v"), (dict(k_out="q"), "k_out overlaps q"),
    (dict(k_out="v"), "k_out overlaps v"), (dict(k_out="q_out"), "k_out overlaps q_out"),
    (dict(k_cache="q"), "k_cache overlaps q"), (dict(k_cache="k"), "k_cache overlaps k"), (dict(v_cache="v"), "v_cache overlaps v"),
    (dict(v_cache="k_cache"), "v_cache overlaps k_cache"), (dict(v_cache="q_out"), "v_cache overlaps q_out"),
    (dict(k_cache="k_out"), "k_cache overlaps k_out"), (dict(q_out="positions"), "q_out overlaps positions"),
    (dict(q_out="cos_sin"), "q_out overlaps cos_sin"), (dict(k_out="slot_map"), "k_out overlaps slot_map"),
    (dict(q_out="q_weight"), "q_out overlaps q_weight"), (dict(k_cache="k_weight"), "k_cache overlaps k_weight"),
])
def test_forward_refuses(kw, what):
    code, text = forward(**{n: AT[m] for n, m in kw.items()})
    assert code == INVALID and what in text.decode()


@pytest.mark.parametrize("kw,what", [
    (dict(dq="k"), "dq overlaps k"), (dict(dq="dk_out"), "dq overlaps dk_out"), (dict(dk="q"), "dk overlaps q"),
    (dict(dk="dq_out"), "dk overlaps dq_out"), (dict(dk="dq"), "dk overlaps dq"), (dict(workspace="dq_out"), "workspace overlaps dq_out"),
    (dict(workspace="dq"), "workspace overlaps dq"), (dict(workspace="q"), "workspace overlaps q"),
    (dict(dq_weight="dk"), "dq_weight overlaps dk"), (dict(dk_weight="dq_weight"), "dk_weight overlaps dq_weight"),
    (dict(dk_weight="workspace"), "workspace overlaps dk_weight"), (dict(dq_weight="q_weight"), "dq_weight overlaps q_weight"),
    (dict(dq="positions"), "dq overlaps positions"), (dict(dk="cos_sin"), "dk overlaps cos_sin"),
])
def test_backward_refuses(kw, what):
    code, text = backward(**{n: AT[m] for n, m in kw.items()})
    assert code == INVALID and what in text.decode()


def test_in_place_with_other_strides_or_some_rows_on_is_refused():
    packed = (2 * HQ * D, D)
    for call, out in ((forward, "q_out"), (backward, "dq")):
        for kw in (dict(strides={"q": packed}), dict(strides={out: packed}), dict(q=AT["q"] + ROW), dict(q=AT["q"] + HQ * ROW),
                   dict(q=AT["q"] + 16), dict(q=AT["q"] + T * HQ * ROW - 16)):
            code, text = call(**{out: AT["q"], **kw})
            assert code == INVALID and f"{out} overlaps q" in text.decode()
        assert call(**{out: AT["q"], "q": AT["q"] + T * HQ * ROW})[0] == STOPPED     # right behind it
    # an extent that no address space holds
    assert forward(q=paged.Heads(AT["q"], 1 << 61, D), q_out=AT["q"] + (1 << 30))[0] == INVALID


def test_rows_between_rows_against_counting():
    # random layouts of two results in one buffer: refused exactly where two rows meet if their strides are the
    # same, and there at least if they are not
    rng = np.random.default_rng(0)
    seen = {True: 0, False: 0}
    for i in range(3000):
        n, hq, hkv = (int(x) for x in rng.integers(1, 6, 3))
        unit = 8                              # elements of 16 bytes
        def layout():  # noqa: E306
            a, b = D + unit * int(rng.integers(0, 40)), D * int(rng.integers(1, 5)) + unit * int(rng.integers(0, 3))
            a = a if rng.random() < 0.5 else D * int(rng.integers(1, 25))
            return (a, b) if rng.random() < 0.5 else (b, a)
        sq = layout()
        sk = sq if rng.random() < 0.7 else layout()
        k_at = AT["q_out"] + 16 * int(rng.integers(-40, 400))
        rows = [{at + 2 * (t * s[0] + h * s[1]) + 16 * x for t in range(n) for h in range(H) for x in range(ROW // 16)}
                for at, s, H in ((AT["q_out"], sq, hq), (k_at, sk, hkv))]
        if any(len(r) != n * H * ROW // 16 for r, H in zip(rows, (hq, hkv))):
            continue                          # rows of one result on one another: refused before
        meet = bool(rows[0] & rows[1])
        code, text = forward({"q_out": sq, "k_out": sk}, T=n, Hq=hq, Hkv=hkv, k_out=k_at)
        if code == INVALID and b"overlapping rows" in text:
            continue                          # (that check knows whole tokens or whole heads apart only)
        if sq == sk:
            assert (code == INVALID) == meet, (n, hq, hkv, sq, sk, hex(k_at))
            seen[meet] += 1
        elif meet:
            assert code == INVALID, (n, hq, hkv, sq, sk, hex(k_at))
    assert min(seen.values()) > 100


# ---- attention --------------------------------------------------------------------------

R, MAX_PAGES, STRIDE = 4, 8, 9
PREFIX = 100
ATTN_AT = dict(q=0x1000000, k_cache=0x2000000, v_cache=0x3000000, out=0x4000000, lse=0x5000000, cu_q=0x5100000, kv_len=0x5200000,
               block_table=0x5300000, prefix_pages=0x5400000, workspace=0x10000000)


def attention(prefix=PREFIX, **kw):
    a = {**ATTN_AT, **kw}
    return stopped(lambda lib: lib.rsa_prefix_attn_fwd(a["q"], HQ * D, D, a["k_cache"], a["v_cache"], 1, T, HQ, HKV, D, PAGE, PAGES,
                                                       a["cu_q"], a["kv_len"], R, a["block_table"], STRIDE, MAX_PAGES,
                                                       a["prefix_pages"], prefix, a["out"], a["lse"], a["workspace"], 1 << 30, None))


@pytest.mark.parametrize("out", ["out", "lse", "workspace"])
@pytest.mark.parametrize("index,entries", [("cu_q", R + 1), ("kv_len", R), ("block_table", (R - 1) * STRIDE + MAX_PAGES),
                                           ("prefix_pages", -(-PREFIX // PAGE))])
def test_attention_refuses_results_over_its_lengths_and_tables(out, index, entries):
    code, text = attention(**{index: ATTN_AT[out]})
    assert code == INVALID and f"{out} overlaps {index}" in text.decode()
    code, text = attention(**{index: ATTN_AT[out] - 4 * (entries - 1)})       # its last entry
    assert code == INVALID and f"{out} overlaps {index}" in text.decode()
    assert attention(**{index: ATTN_AT[out] - 4 * entries})[0] == STOPPED     # right before


def test_attention_takes_operands_of_their_own():
    assert attention()[0] == STOPPED
    assert attention(cu_q=ATTN_AT["kv_len"])[0] == STOPPED                    # only read
    assert attention(prefix=0, prefix_pages=ATTN_AT["out"])[0] == STOPPED     # not read


@pytest.mark.parametrize("n", [29, 30, 31, 62])
def test_attention_workspace_has_a_plan_of_requests_and_two_words(n):
    # 8 bytes each, rounded up to 256: 30 requests are the most that one such unit holds
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    rest = 2 * (up(T * HQ * D * 4) + up(T * HQ * 4)) + up(160 * 256 * D * 4) + up(160 * 256 * 4)
    assert rsa.prefix_attn_workspace_size(torch.bfloat16, T, HQ, HKV, D, n) == up((n + 2) * 8) + rest
