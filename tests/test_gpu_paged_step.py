"""The paged-cache operators together, as a server runs them: a prompt's step,
then captured decode steps, the plan feeding the cache write and the attention;
the cache grows page by page behind a shared prefix.  Compared with attention
over dense keys in 64 bits."""
import threading

import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,page,prefix,pad", [(torch.bfloat16, 128, 16, 150, 3), (torch.bfloat16, 64, 64, 0, 0),
                                                     (torch.float32, 64, 32, 33, 2)])
def test_prompt_then_captured_decode(dtype, d, page, prefix, pad):
    need_cuda()
    g = torch.Generator().manual_seed(d + prefix)
    R, Hq, Hkv, max_pages, n_pages = 4, 6, 2, 6, 60
    prompts, steps = [5, 1, 30, page], 2 * 9
    rows = R + pad
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    cs = rsa.rope_table(prefix + 200, d)
    kc, vc = (torch.full((n_pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    free = torch.randperm(n_pages, generator=g).to(torch.int32)
    npre = -(-prefix // page)
    prefix_pages, free = free[:npre].cuda(), free[npre:].cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def project(n):
        """A step's packed q, k, v rows."""
        return torch.randn(n, (Hq + 2 * Hkv) * d, generator=g).to(dtype)

    def cut(x):
        n = x.shape[0]
        return (x[:, :Hq * d].view(n, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(n, Hkv, d), x[:, (Hq + Hkv) * d:].view(n, Hkv, d))

    seen = [[] for _ in range(R)]  # every request's (k, v) rows in 64 bits, as written to the cache
    pre = None
    if prefix:
        # the shared document: one sequence of its own
        x = project(prefix).cuda()
        q, k, v = cut(x)
        t = torch.arange(prefix, device="cuda")
        ko = torch.empty(prefix, Hkv, d, dtype=dtype, device="cuda")
        rsa.qk_norm_rope(q, k, wq, wk, t, cs, v=v, slot_map=prefix_pages[t // page].long() * page + t % page, k_cache=kc,
                         v_cache=vc, k_out=ko)
        pre = ref.to64(ko), ref.to64(v)

    table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")

    def step(x, plan, ko=None):
        q, k, v = cut(x)
        qo, _ = rsa.qk_norm_rope(q, k, wq, wk, plan.positions, cs, v=v, slot_map=plan.slot_map, k_cache=kc, v_cache=vc, k_out=ko)
        out, lse = rsa.prefix_attn(qo, kc, vc, plan.cu_new, table, plan.kv_len, prefix_pages=prefix_pages, prefix_len=prefix)
        return qo, out, lse

    def check(qo, ko, v, out, lse, cu, lens):
        """The newest rows against dense attention over what was written."""
        for r in range(R):
            for i in range(cu[r], cu[r + 1]):
                seen[r].append((ref.to64(ko[i]), ref.to64(v[i])))
        kd, vd = (np.concatenate(([pre[c]] if prefix else []) + [np.stack([y[c] for y in s]) for s in seen]) for c in (0, 1))
        # one page of one row for each token: a dense view of the same keys
        pages = lambda n, at: np.arange(at, at + n)  # noqa: E731
        dense_table = np.zeros((R, max(lens)), np.int64)
        at = prefix
        for r in range(R):
            dense_table[r, :lens[r]] = pages(lens[r], at)
            at += lens[r]
        rr = ref.prefix_attn(ref.to64(qo), kd[:, :, None], vd[:, :, None], cu, dense_table, lens, pages(prefix, 0), prefix)
        ref.assert_prefix_attn(out, lse, rr, dtype, cu[R])

    x = project(sum(prompts)).cuda()
    plan = rsa.page_plan(i32([0] * R), i32(prompts), table, free, page, n_pages, sum(prompts), pos0=prefix)
    ko = torch.empty(sum(prompts), Hkv, d, dtype=dtype, device="cuda")
    qo, out, lse = step(x, plan, ko)
    lens = list(prompts)
    cu = plan.cu_new.tolist()
    assert plan.info[0].item() == 0
    check(qo, ko, cut(x)[2], out, lse, cu, lens)

    # decode: one token a request, two steps a replay, the plans' buffers taking turns; request 1 stops half way
    x = project(rows).cuda()
    new = lambda: rsa.PagePlan(torch.empty(R + 1, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda"),  # noqa: E731
                               *(torch.empty(n, dtype=torch.int64, device="cuda") for n in (rows, rows, 4)))
    a, b = new(), new()
    b.kv_len.copy_(plan.kv_len)
    b.info.copy_(plan.info)
    one = i32([1] * R)
    ko = torch.empty(rows, Hkv, d, dtype=dtype, device="cuda")
    kv = (kc, vc)
    saved = [t.clone() for t in (*kv, table)]

    def turn(frm, to):
        rsa.page_plan(frm.kv_len, one, table, free, page, n_pages, rows, free_start=frm.info[3:], pos0=prefix, out=to)
        return step(x, to, ko)
    turn(b, a)  # warm: every kernel loaded before the capture
    torch.cuda.synchronize()
    for t, s in zip((*kv, table), saved):
        t.copy_(s)
    graphs = []
    for frm, to in ((b, a), (a, b)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = turn(frm, to)
        graphs.append((gr, to, res))
    for i in range(steps):
        if i == steps // 2:
            one.copy_(i32([1, 0, 1, 1]))
        x.copy_(project(rows))
        gr, to, (qo, out, lse) = graphs[i % 2]
        out.fill_(3)
        gr.replay()
        torch.cuda.synchronize()
        assert to.info[0].item() == 0
        cu = to.cu_new.tolist()
        lens = to.kv_len.tolist()
        if i in (0, 1, 11, steps - 1):
            check(qo, ko, cut(x)[2], out, lse, cu, lens)
            assert (out[cu[R]:] == 3).all()
        else:
            for r in range(R):
                for j in range(cu[r], cu[r + 1]):
                    seen[r].append((ref.to64(ko[j]), ref.to64(cut(x)[2][j])))
        assert [len(s) for s in seen] == lens
    rsa.check_device_error()


def test_outputs_made_for_another_stream_wait_for_their_memory():
    # The memory of a tensor that the current stream still reads may be handed out for a call's outputs: a call on
    # another stream must not write it before that reading is done.
    need_cuda()
    T, H, d = 4096, 8, 128
    k = torch.randn(T, H, d, device="cuda")
    x = torch.full((T, H, d), 7.0, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)   # some ten milliseconds on the current stream
    y = x.clone()
    at = x.data_ptr()
    del x
    q, _ = rsa.qk_norm_rope(k, k, None, None, None, None, stream=side)
    assert q.data_ptr() == at       # (the block came back at once: else this shows nothing)
    torch.cuda.synchronize()
    assert (y == 7).all()


def test_host_tensors_are_refused_with_a_gpu_at_hand():
    need_cuda()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):
        rsa.page_plan(i32(2), i32(2), i32(2, 2), i32(4), 16, 4, 8)
    with pytest.raises(TypeError):
        rsa.page_plan(i32(2).cuda(), i32(2), i32(2, 2).cuda(), i32(4).cuda(), 16, 4, 8)
    x = torch.zeros(2, 2, 64, device="cuda")
    with pytest.raises(TypeError):
        rsa.qk_norm_rope(x, x.cpu(), None, None, None, None)
    with pytest.raises(TypeError):
        rsa.prefix_attn(x, x.view(1, 2, 1, 128).cpu(), x, i32(3), i32(2, 1), i32(2))


def test_calls_of_two_threads_at_once():
    # the calls let go of the interpreter while they launch; each thread has its stream and gets its own results
    need_cuda()
    T, Hq, Hkv, d, page = 40, 8, 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = rand(60, Hkv, page, d), rand(60, Hkv, page, d)
    cu, lens = i32(list(range(T + 1))), i32([1 + i for i in range(T)])
    table = torch.arange(T * 2, device="cuda").view(T, 2).to(torch.int32) % 60
    qs, cos_sin, pos = [rand(T, Hq, d) for _ in range(2)], rsa.rope_table(100, d), torch.arange(T, device="cuda")

    def step(q):
        x, _ = rsa.qk_norm_rope(q, q[:, :2], None, None, pos, cos_sin)
        return rsa.prefix_attn(x, kc, vc, cu, table, lens, prefix_pages=table[3], prefix_len=50)
    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    got[i].append(step(qs[i]))
                    del got[i][:-3]
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    rsa.check_device_error()


def test_arguments_that_are_no_fitting_objects():
    need_cuda()
    q = torch.randn(3, 4, 64, device="cuda")
    kc = torch.randn(4, 2, 16, 64, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q, kc, kc.clone(), i32(0, 1, 3), torch.zeros(2, 2, dtype=torch.int32, device="cuda"), i32(5, 7))
    out, lse = rsa.prefix_attn(*args)
    n = rsa.prefix_attn_workspace_size(torch.float32, 3, 4, 2, 64, 2)
    for bad, err in [(dict(stream=object()), TypeError), (dict(stream="0"), TypeError), (dict(prefix_len=1.5), TypeError),
                     (dict(prefix_len=-1, prefix_pages=i32(0)), rsa.RsaError), (dict(prefix_len=10), TypeError),
                     (dict(workspace=torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]), ValueError),
                     (dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n)), ValueError),
                     (dict(workspace=torch.zeros(n, dtype=torch.uint8)), TypeError), (dict(out=q.data_ptr()), TypeError),
                     (dict(out=q), rsa.RsaError), (dict(lse=lse.t().contiguous().t()), ValueError)]:
        with pytest.raises(err):
            rsa.prefix_attn(*args, **bad)
    pos, table = torch.arange(3, device="cuda"), rsa.rope_table(10, 64)
    for bad, err in [(dict(sections=5), TypeError), (dict(sections=[]), ValueError), (dict(sections=[8] * 5), ValueError),
                     (dict(sections=["a"]), TypeError), (dict(eps="x"), TypeError), (dict(eps=float("nan")), rsa.RsaError),
                     (dict(eps=-1.0), rsa.RsaError)]:
        with pytest.raises(err):
            rsa.qk_norm_rope(q, q, None, None, pos, table, **bad)
    with pytest.raises(TypeError):
        rsa.qk_norm_rope(q, q, None, None, None, table)
    # leaves of a graph are read like any tensor, and results have no history
    leaf = torch.nn.Parameter(q)
    a, b = rsa.qk_norm_rope(leaf, leaf, None, None, pos, table)
    assert not a.requires_grad and torch.equal(a, rsa.qk_norm_rope(q, q, None, None, pos, table)[0])
    out2, lse2 = rsa.prefix_attn(*args, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert rsa.prefix_attn(*args, out=out2, lse=lse2)[0] is out2
    rsa.check_device_error()
